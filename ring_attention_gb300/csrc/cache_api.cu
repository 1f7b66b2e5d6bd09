// cache_api.cu - the C entry points of the paged 8-bit cache (declared in include/bpa.h):
// argument checks, workspace and launches.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <nvtx3/nvToolsExt.h>

#include "bpa.h"
#include "bpa_internal.h"
#include "cache.h"

using namespace bpa;

namespace {

constexpr size_t kHeader = 256;                  // the status word
constexpr int64_t kMost = int64_t{1} << 30;      // rows, tokens of the cache, tokens of a table row

bpa_status fail(bpa_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    set_last_error(buf);
    return st;
}

struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange&) = delete;
    NvtxRange& operator=(const NvtxRange&) = delete;
};

bpa_status cuda_status(cudaError_t e, const char* what) {
    return e == cudaSuccess ? BPA_OK : fail(BPA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

bpa_status check_ws(const void* ws, size_t have, size_t need) {
    if (!ws) return fail(BPA_ERR_WORKSPACE, "workspace is NULL (need %zu bytes)", need);
    if (reinterpret_cast<uintptr_t>(ws) & 255u) return fail(BPA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    if (have < need) return fail(BPA_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", have, need);
    return BPA_OK;
}

bpa_status check_paging(int32_t page_size, int32_t num_pages) {
    if (page_size < 1 || page_size > 1024) return fail(BPA_ERR_INVALID_ARG, "page_size %d outside [1, 1024]", page_size);
    if (num_pages < 1 || static_cast<int64_t>(num_pages) * page_size > kMost)
        return fail(BPA_ERR_INVALID_ARG, "%d pages of %d tokens: need 1 to 2^30 tokens", num_pages, page_size);
    return BPA_OK;
}

bpa_status check_table(int32_t page_size, int32_t max_pages) {
    if (max_pages < 1 || static_cast<int64_t>(max_pages) * page_size > kMost)
        return fail(BPA_ERR_INVALID_ARG, "max_pages %d of %d tokens: need 1 to 2^30 tokens", max_pages, page_size);
    return BPA_OK;
}

// dv resolved; pointers are not looked at
bpa_status check_cache(const bpa_cache_desc* c, int& dv) {
    if (!c) return fail(BPA_ERR_INVALID_ARG, "cache descriptor is NULL");
    if (c->struct_size != sizeof(bpa_cache_desc))
        return fail(BPA_ERR_INVALID_ARG, "cache->struct_size is %u, expected %zu", c->struct_size, sizeof(bpa_cache_desc));
    if (c->dtype != BPA_BF16 && c->dtype != BPA_FP32) return fail(BPA_ERR_INVALID_ARG, "unknown dtype %d", c->dtype);
    if (c->reserved) return fail(BPA_ERR_INVALID_ARG, "cache->reserved must be 0");
    dv = c->dv ? c->dv : c->d;
    if (c->Hkv < 1 || c->d < 1 || dv < 1) return fail(BPA_ERR_INVALID_ARG, "Hkv, d must be >= 1, dv >= 0");
    if (c->d > 512 || dv > 512) return fail(BPA_ERR_UNSUPPORTED, "head dims %d, %d: at most 512", c->d, dv);
    if (c->Hkv > 65535) return fail(BPA_ERR_UNSUPPORTED, "%d kv heads, more than 65535", c->Hkv);
    for (int i = 0; i < 3; ++i)
        if (c->k_cache_strides[i] < 0 || c->v_cache_strides[i] < 0)
            return fail(BPA_ERR_INVALID_ARG, "cache strides must be >= 0");
    return check_paging(c->page_size, c->num_pages);
}

bpa_status check_cache_pointers(const bpa_cache_desc* c) {
    if (!c->k_cache || !c->v_cache || !c->k_scale || !c->v_scale)
        return fail(BPA_ERR_INVALID_ARG, "k_cache, v_cache, k_scale or v_scale is NULL");
    return BPA_OK;
}

// A cache as a 4-D map (channel, token, head, page) of bytes; false where its layout does not suit TMA
// (16-byte aligned base, strides in multiples of 16 bytes).
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

bool make_cache_map(CUtensorMap* map, const uint8_t* base, const CacheAttnArgs& a, int channels, const int64_t st[3],
                    int box_cols, int box_rows, bool swizzled) {
    static const EncodeTiledFn enc = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                            cudaSuccess && q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<EncodeTiledFn>(p) : nullptr;
    }();
    if (!enc || (reinterpret_cast<uintptr_t>(base) & 15)) return false;
    const int extent[3] = {a.P, a.Hkv, a.num_pages};
    const int64_t given[3] = {st[2], st[1], st[0]};
    cuuint64_t dims[4] = {static_cast<cuuint64_t>(channels), static_cast<cuuint64_t>(a.P),
                          static_cast<cuuint64_t>(a.Hkv), static_cast<cuuint64_t>(a.num_pages)};
    cuuint64_t strides[3];
    for (int i = 0; i < 3; ++i) {
        const int64_t s = extent[i] == 1 ? 16 : given[i];   // a dimension of extent 1 never steps
        if (s < 16 || s % 16 || s >= int64_t{1} << 40) return false;
        strides[i] = static_cast<cuuint64_t>(s);
    }
    cuuint32_t box[4] = {static_cast<cuuint32_t>(box_cols), static_cast<cuuint32_t>(box_rows), 1, 1};
    cuuint32_t one[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t*>(base), dims, strides, box, one,
               CU_TENSOR_MAP_INTERLEAVE_NONE,
               !swizzled ? CU_TENSOR_MAP_SWIZZLE_NONE : box_cols == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bpa_status make_attn(const bpa_cache_desc* c, const bpa_cache_batch* b, CacheAttnArgs& a) {
    int dv = 0;
    bpa_status st = check_cache(c, dv);
    if (st != BPA_OK) return st;
    if (!b) return fail(BPA_ERR_INVALID_ARG, "batch descriptor is NULL");
    if (b->struct_size != sizeof(bpa_cache_batch))
        return fail(BPA_ERR_INVALID_ARG, "batch->struct_size is %u, expected %zu", b->struct_size,
                    sizeof(bpa_cache_batch));
    if (b->R < 1 || b->T < 0 || b->T > kMost) return fail(BPA_ERR_INVALID_ARG, "need R >= 1, 0 <= T <= 2^30");
    if (b->Hq < 1 || b->Hq % c->Hkv)
        return fail(BPA_ERR_INVALID_ARG, "Hq (%d) must be a multiple of Hkv (%d)", b->Hq, c->Hkv);
    if (b->Hq > 65535) return fail(BPA_ERR_UNSUPPORTED, "%d q heads, more than 65535", b->Hq);
    if (b->max_q < 0) return fail(BPA_ERR_INVALID_ARG, "max_q must be >= 0");
    if ((st = check_table(c->page_size, b->max_pages)) != BPA_OK) return st;
    if (b->window_left < -1 || b->window_right < -1)
        return fail(BPA_ERR_INVALID_ARG, "window bounds must be >= -1");
    for (int i = 0; i < 2; ++i)
        if (b->q_strides[i] < 0 || b->o_strides[i] < 0) return fail(BPA_ERR_INVALID_ARG, "strides must be >= 0");
    memset(&a, 0, sizeof a);
    a.dtype = c->dtype;
    a.R = b->R;
    a.T = b->T;
    a.Hq = b->Hq;
    a.Hkv = c->Hkv;
    a.G = b->Hq / c->Hkv;
    a.d = c->d;
    a.dv = dv;
    a.P = c->page_size;
    a.num_pages = c->num_pages;
    a.max_pages = b->max_pages;
    a.max_q = b->max_q && b->max_q < b->T ? b->max_q : b->T;
    a.scale = b->scale > 0.f ? b->scale : 1.f / sqrtf(static_cast<float>(c->d));
    a.causal = b->causal != 0;
    a.wl = b->window_left;
    a.wr = b->window_right;
    a.q = b->q;
    a.kc = static_cast<const uint8_t*>(c->k_cache);
    a.vc = static_cast<const uint8_t*>(c->v_cache);
    for (int i = 0; i < 2; ++i) {
        a.qs[i] = b->q_strides[i];
        a.os[i] = b->o_strides[i];
    }
    for (int i = 0; i < 3; ++i) {
        a.kcs[i] = c->k_cache_strides[i];
        a.vcs[i] = c->v_cache_strides[i];
    }
    a.kscale = c->k_scale;
    a.vscale = c->v_scale;
    a.table = b->page_table;
    a.kv_lens = b->kv_lens;
    a.cu_q = b->cu_q;
    a.sink = b->sink;
    return BPA_OK;
}

}  // namespace

extern "C" {

bpa_status bpa_cache_plan(int32_t R, int32_t T, int32_t page_size, int32_t num_pages, int32_t max_pages,
                          const int32_t* ctx_lens, const int32_t* new_lens, const int32_t* free_pages,
                          const int32_t* free_count, int32_t* page_table, int32_t* kv_lens, int32_t* cu_q,
                          int32_t* slot_map, int32_t* positions, int32_t* ctx_lens_out, int32_t* free_count_out,
                          void* workspace, size_t workspace_bytes, void* stream) {
    const NvtxRange range("bpa_cache_plan");
    if (R < 1 || T < 0 || T > kMost) return fail(BPA_ERR_INVALID_ARG, "need R >= 1, 0 <= T <= 2^30");
    if (R > kPlanMaxR) return fail(BPA_ERR_UNSUPPORTED, "%d requests, more than %d", R, kPlanMaxR);
    bpa_status st = check_paging(page_size, num_pages);
    if (st != BPA_OK || (st = check_table(page_size, max_pages)) != BPA_OK) return st;
    if (!ctx_lens || !new_lens || !free_pages || !free_count || !page_table || !kv_lens || !cu_q || !ctx_lens_out ||
        !free_count_out || (!slot_map && T))
        return fail(BPA_ERR_INVALID_ARG, "a buffer other than positions is NULL");
    if ((st = check_ws(workspace, workspace_bytes, kHeader)) != BPA_OK) return st;
    PlanArgs a = {R, T, page_size, num_pages, max_pages, ctx_lens, new_lens, free_pages, free_count, page_table,
                  kv_lens, cu_q, slot_map, positions, ctx_lens_out, free_count_out,
                  static_cast<uint32_t*>(workspace)};
    return cuda_status(launch_cache_plan(a, static_cast<cudaStream_t>(stream)), "plan launch");
}

bpa_status bpa_cache_append(const bpa_cache_desc* cache, const void* k, const void* v, const int64_t k_strides[2],
                            const int64_t v_strides[2], const int32_t* slot_map, int32_t T, int32_t max_new,
                            void* workspace, size_t workspace_bytes, void* stream) {
    const NvtxRange range("bpa_cache_append");
    int dv = 0;
    bpa_status st = check_cache(cache, dv);
    if (st != BPA_OK || (st = check_cache_pointers(cache)) != BPA_OK) return st;
    if (T < 0 || T > kMost || max_new < 0) return fail(BPA_ERR_INVALID_ARG, "need 0 <= T <= 2^30, max_new >= 0");
    if (!k_strides || !v_strides || (T && (!k || !v || !slot_map)))
        return fail(BPA_ERR_INVALID_ARG, "k, v, their strides or slot_map is NULL");
    for (int i = 0; i < 2; ++i)
        if (k_strides[i] < 0 || v_strides[i] < 0) return fail(BPA_ERR_INVALID_ARG, "strides must be >= 0");
    const int32_t extents[3] = {cache->num_pages, cache->Hkv, cache->page_size};
    for (int i = 0; i < 3; ++i)
        if (extents[i] > 1 && (cache->k_cache_strides[i] == 0 || cache->v_cache_strides[i] == 0))
            return fail(BPA_ERR_INVALID_ARG, "a cache that is written needs strides above 0");
    if (static_cast<int64_t>(T) * cache->Hkv > kMost)
        return fail(BPA_ERR_UNSUPPORTED, "T * Hkv above 2^30");
    if ((st = check_ws(workspace, workspace_bytes, kHeader)) != BPA_OK) return st;
    AppendArgs a;
    memset(&a, 0, sizeof a);
    a.dtype = cache->dtype;
    a.Hkv = cache->Hkv;
    a.d = cache->d;
    a.dv = dv;
    a.P = cache->page_size;
    a.num_pages = cache->num_pages;
    a.T = T;
    a.k = k;
    a.v = v;
    for (int i = 0; i < 2; ++i) {
        a.ks[i] = k_strides[i];
        a.vs[i] = v_strides[i];
    }
    a.kc = static_cast<uint8_t*>(cache->k_cache);
    a.vc = static_cast<uint8_t*>(cache->v_cache);
    for (int i = 0; i < 3; ++i) {
        a.kcs[i] = cache->k_cache_strides[i];
        a.vcs[i] = cache->v_cache_strides[i];
    }
    a.kscale = cache->k_scale;
    a.vscale = cache->v_scale;
    a.slots = slot_map;
    a.max_new = max_new;
    a.status = static_cast<uint32_t*>(workspace);
    return cuda_status(launch_cache_append(a, static_cast<cudaStream_t>(stream)), "append launch");
}

size_t bpa_cache_attn_workspace_size(const bpa_cache_desc* cache, const bpa_cache_batch* batch) {
    CacheAttnArgs a;
    if (make_attn(cache, batch, a) != BPA_OK) return 0;
    return cache_attn_mma_workspace(a);
}

bpa_status bpa_cache_attn(const bpa_cache_desc* cache, const bpa_cache_batch* batch, void* o, float* m, float* l,
                          void* workspace, size_t workspace_bytes, void* stream) {
    const NvtxRange range("bpa_cache_attn");
    CacheAttnArgs a;
    bpa_status st = make_attn(cache, batch, a);
    if (st != BPA_OK || (st = check_cache_pointers(cache)) != BPA_OK) return st;
    if (!a.table || !a.kv_lens || !a.cu_q || (a.T && (!a.q || !o)))
        return fail(BPA_ERR_INVALID_ARG, "q, o, page_table, kv_lens or cu_q is NULL");
    if (!m != !l) return fail(BPA_ERR_INVALID_ARG, "m and l: both or neither");
    if ((a.T > 1 && a.os[0] == 0) || (a.Hq > 1 && a.os[1] == 0))
        return fail(BPA_ERR_INVALID_ARG, "o_strides must be above 0: rows of o would lie over one another");
    if ((st = check_ws(workspace, workspace_bytes, cache_attn_mma_workspace(a))) != BPA_OK) return st;
    a.o = o;
    a.m = m;
    a.l = l;
    a.status = static_cast<uint32_t*>(workspace);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (a.T > 0 && cache_attn_mma_supported(a)) {
        const CacheBox box = cache_attn_mma_box(a);
        CUtensorMap maps[2];
        if (make_cache_map(&maps[0], a.kc, a, a.d, a.kcs, box.cols_k, box.rows, true) &&
            make_cache_map(&maps[1], a.vc, a, a.dv, a.vcs, box.cols_v, box.rows, true)) {
            uint32_t* far = nullptr;
            if (cache_attn_tc_takes(a)) {               // requests of many rows first
                far = cache_attn_far(static_cast<uint8_t*>(workspace));
                const size_t used = reinterpret_cast<uint8_t*>(far + a.R) - static_cast<uint8_t*>(workspace);
                st = cuda_status(cudaMemsetAsync(workspace, 0, used, s), "clearing the status word and the marks");
                if (st != BPA_OK) return st;
                const CacheBox plain = cache_attn_tc_box(a);
                CUtensorMap raw[2];
                if (!make_cache_map(&raw[0], a.kc, a, a.d, a.kcs, plain.cols_k, plain.rows, false) ||
                    !make_cache_map(&raw[1], a.vc, a, a.dv, a.vcs, plain.cols_v, plain.rows, false))
                    return fail(BPA_ERR_CUDA, "cache attention: no tensor map");
                st = cuda_status(launch_cache_attn_tc(a, raw, a.status + 2, far, s), "cache attention launch");
                if (st != BPA_OK) return st;
            }
            return cuda_status(launch_cache_attn_mma(a, maps, static_cast<uint8_t*>(workspace), far, s),
                               "cache attention launch");
        }
    }
    st = cuda_status(cudaMemsetAsync(workspace, 0, kHeader, s), "clearing the status word");
    if (st != BPA_OK || a.T == 0) return st;
    return cuda_status(launch_cache_attn_simt(a, s), "cache attention launch");
}

}  // extern "C"
