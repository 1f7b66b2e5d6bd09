// cache.h - the paged 8-bit key / value cache: validated calls and kernel launchers of libbpa.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "bpa.h"

namespace bpa {

// Query rows of a kv head up to which a request is one of few rows.  Measured at 64, 32 and 15, requests of
// more going to the tensor cores: 33 requests of 8 to 48 rows (1 to 6 drafted tokens of 8 heads, window
// 1,024) 41.2, 59.9 and 73.4 us; 33 of 8 to 64 rows over up to 8,000 tokens, 128 channels 222, 194 and
// 230.  Pieces of prompts (thousands of rows) take 1,540 us there and 7.1 ms here.
constexpr int kFewRows = 64;
// The same under a tree, where the tensor cores share out keys as well: 19 requests of 8,192 tokens, 4 q heads a kv
// head, 128 channels; 64 rows 138 us there and 249 here, 32 rows 137 and 142.
constexpr int kFewTreeRows = 32;
constexpr int kPlanMaxR = 8192;      // requests of one plan: their lengths and offsets sit in shared memory
constexpr int kMaxTreeWords = 32;    // words of a row's mask: 1,024 rows of a request

struct PlanArgs {
    int R, T, P, num_pages, max_pages;
    const int32_t *ctx, *add, *free_pages, *free_count;
    int32_t *table, *kv_lens, *cu_q, *slots, *positions, *ctx_out, *count_out;
    uint32_t* status;
};

struct AppendArgs {
    int dtype, Hkv, d, dv, P, num_pages, T;
    const void *k, *v;
    int64_t ks[2], vs[2];            // (row, head) strides
    uint8_t *kc, *vc;
    int64_t kcs[3], vcs[3];          // (page, head, token) strides
    float *kscale, *vscale;          // [num_pages, Hkv]
    const int32_t* slots;
    int max_new;
    uint32_t* status;
};

struct TreeArgs {
    int R, T, words;
    int wl;                          // ancestors up to this many steps above a row are in its mask; -1: all
    const int32_t *parents, *kv_lens, *cu_q;
    uint32_t* tree;                  // [T, words]
    int32_t* positions;              // [T]
    uint32_t* status;
};

struct KeepArgs {
    int R, T, Hkv, d, dv, P, num_pages, max_pages, max_keep;
    uint8_t *kc, *vc;
    int64_t kcs[3], vcs[3];          // (page, head, token) strides
    float *kscale, *vscale;          // [num_pages, Hkv]
    const int32_t *table, *kv_lens, *cu_q, *keep, *count;
    uint32_t* status;
};

struct ForkArgs {
    int N, R, P, num_pages, max_pages;
    const int32_t *src, *dst, *ctx;
    int32_t *table, *refs;
    const int32_t *free_pages, *free_count;
    int32_t *copy_src, *copy_dst, *ctx_out, *count_out;
    uint32_t* status;
};

struct ReleaseArgs {
    int R, P, num_pages, max_pages;
    const int32_t *ctx, *keep, *table;
    int32_t *refs, *free_pages;
    const int32_t* free_count;
    int32_t *ctx_out, *count_out;
    uint32_t* status;
};

struct CopyArgs {
    int N, Hkv, d, dv, P, num_pages;
    uint8_t *kc, *vc;
    int64_t kcs[3], vcs[3];
    float *kscale, *vscale;
    const int32_t *src, *dst;
    uint32_t* status;
};

struct CacheAttnArgs {
    int dtype, R, T, Hq, Hkv, G, d, dv, P, num_pages, max_pages, max_q;
    float scale;
    int causal, wl, wr;              // wl, wr: -1 = unbounded
    const void* q;
    int64_t qs[2], os[2];            // (row, head) strides
    void* o;
    float *m, *l;                    // [Hq, T] or null
    const uint8_t *kc, *vc;
    int64_t kcs[3], vcs[3];
    const float *kscale, *vscale;
    const int32_t *table, *kv_lens, *cu_q;
    const float* sink;
    const uint32_t* tree;            // [T, tree_words] masks over a request's own rows, or null
    int tree_words;
    uint32_t* status;
};

namespace cache_mma {
struct Pieces;                       // cache_pieces.h
}

#ifdef __CUDACC__
// Programmatic dependent launch: a kernel launched by launch_early is set up while the one before it
// on the stream ends; it calls wait_for_previous() before it touches anything in global memory (with
// plain loads, which the compiler does not move across it, until an address depends on one), so the
// stream's order holds for everything that a caller can see.  No kernel here lets the next one start
// before its own end: measured, CTAs of the next kernel then take room on some SMs while the join
// still runs there, and a persistent kernel that is not spread evenly cost 64 requests x up to 8192
// tokens 135 us instead of 100.
__device__ __forceinline__ void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
cudaError_t launch_early(dim3 grid, dim3 block, size_t smem, cudaStream_t s, void (*kernel)(P...), A... args) {
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

// Rows and keys of request r, made safe to address: rows clamped to [0, T], the length to the table.
struct Req {
    int row0, n, len;                // first packed row, rows, keys
    bool bad;                        // the length did not fit
};
__device__ __forceinline__ Req request_of(const CacheAttnArgs& a, int r) {
    Req q;
    q.row0 = min(max(*(a.cu_q + r), 0), a.T);
    q.n = max(min(*(a.cu_q + r + 1), a.T) - q.row0, 0);
    const int64_t cap = static_cast<int64_t>(a.max_pages) * a.P;
    const int len = *(a.kv_lens + r);
    q.len = static_cast<int>(min(static_cast<int64_t>(max(len, 0)), cap));
    q.bad = len != q.len;
    return q;
}
// Keys [lo, hi] that the masks leave row i of a request (empty: lo > hi).
__device__ __forceinline__ void row_keys(const CacheAttnArgs& a, const Req& q, int i, int& lo, int& hi) {
    const int p = q.len - q.n + i;
    lo = 0;
    hi = q.len - 1;
    if (a.causal) hi = min(hi, p);
    if (a.wr >= 0) hi = static_cast<int>(min(static_cast<int64_t>(hi), static_cast<int64_t>(p) + a.wr));
    if (a.wl >= 0) lo = static_cast<int>(max(static_cast<int64_t>(0), static_cast<int64_t>(p) - a.wl));
}

// The same under a tree: of the tokens in front of the step's, those from lo on; of the step's own, those whose
// bit the row's mask has.
struct TreeRow {
    int lo, ctx;                     // first key of the window, tokens in front of the step's (may be negative)
    const uint32_t* bits;
    int words;
    __device__ __forceinline__ bool allows(int k) const {
        if (k < ctx) return k >= lo;
        const int64_t j = static_cast<int64_t>(k) - ctx;
        return j < 32 * static_cast<int64_t>(words) && (__ldg(bits + (j >> 5)) >> (j & 31) & 1);
    }
};
__device__ __forceinline__ TreeRow tree_row(const CacheAttnArgs& a, const Req& q, int i) {
    TreeRow t = {0, q.len - q.n, a.tree + static_cast<int64_t>(q.row0 + i) * a.tree_words, a.tree_words};
    if (a.wl >= 0) {                 // the row stands as deep as it has ancestors among the step's tokens
        int depth = 0;
        for (int w = 0; w < t.words && 32 * w < i; ++w) {
            const uint32_t before = i - 32 * w >= 32 ? 0xffffffffu : (1u << (i - 32 * w)) - 1;
            depth += __popc(__ldg(t.bits + w) & before);
        }
        t.lo = static_cast<int>(max(static_cast<int64_t>(0), static_cast<int64_t>(t.ctx) + depth - a.wl));
    }
    return t;
}
// Keys [lo, hi] that hold whatever the rows of a request see under a tree (empty: lo > hi).
__device__ __forceinline__ void tree_span(const CacheAttnArgs& a, const Req& q, int& lo, int& hi) {
    const int ctx = max(q.len - q.n, 0);
    lo = a.wl >= 0 ? static_cast<int>(max(static_cast<int64_t>(0), static_cast<int64_t>(ctx) - a.wl)) : 0;
    hi = q.len - 1;
}
#endif

cudaError_t launch_cache_plan(const PlanArgs& a, cudaStream_t s);
cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t s);
cudaError_t launch_cache_tree(const TreeArgs& a, cudaStream_t s);             // status word clear
cudaError_t launch_cache_keep(const KeepArgs& a, cudaStream_t s);             // status word clear
cudaError_t launch_cache_fork(const ForkArgs& a, cudaStream_t s);
cudaError_t launch_cache_release(const ReleaseArgs& a, cudaStream_t s);
cudaError_t launch_cache_copy(const CopyArgs& a, cudaStream_t s);
cudaError_t launch_cache_attn_simt(const CacheAttnArgs& a, cudaStream_t s);   // any shape

// Matrix-instruction kernels for few rows: head dims in steps of 16 up to 256, pages of 16, 32 or a
// multiple of 64 tokens; they read the cache through tensor maps (channel, token, head, page) with
// boxes of `cols_k` / `cols_v` channels and `rows` tokens.
struct CacheBox {
    int cols_k, cols_v, rows;
};
bool cache_attn_mma_supported(const CacheAttnArgs& a);
size_t cache_attn_mma_workspace(const CacheAttnArgs& a);
CacheBox cache_attn_mma_box(const CacheAttnArgs& a);
// far: null, or the marks of launch_cache_attn_tc, which has run before on the same status word: requests
// of more than kFewRows rows are then computed only where they are marked.
// more: null, or pieces that launch_cache_attn_tc has left for the join (trees).
cudaError_t launch_cache_attn_mma(const CacheAttnArgs& a, const CUtensorMap* maps, uint8_t* ws, const uint32_t* far,
                                  const cache_mma::Pieces* more, cudaStream_t s);
uint32_t* cache_attn_far(uint8_t* ws);      // the marks' place, [R]

// Tensor-core kernel for requests of more than kFewRows rows (bf16, head dims in steps of 16 up to 128,
// pages in steps of 16 tokens); the others are left alone.  counter, far [R]: zero before the launch; it marks
// the requests whose v scales lie too far apart for it, whatever it has written for them.
bool cache_attn_tc_takes(const CacheAttnArgs& a);       // supported, and there may be enough such requests
CacheBox cache_attn_tc_box(const CacheAttnArgs& a);      // plain (not swizzled) boxes
// ws: of trees, cache_attn_tc_workspace bytes; *left: their pieces, for the join.
cudaError_t launch_cache_attn_tc(const CacheAttnArgs& a, const CUtensorMap* maps, uint32_t* counter, uint32_t* far, uint8_t* ws, cache_mma::Pieces* left, cudaStream_t s);
size_t cache_attn_tc_workspace(const CacheAttnArgs& a);

}  // namespace bpa
