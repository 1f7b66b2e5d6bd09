// cache_pages.cu - pages of the 8-bit cache shared, copied and given back, on the device.
//
// page_refs[page] counts a page's holders beyond the first.  A fork takes its parent's full pages (one more
// holder each) and a page of its own for the last one, if that is not full, so a page that is still
// written has one holder.  A release takes a holder from each page that a request gives up; a page without
// any left (its count went to -1) goes to the end of the free list, in ascending order of ids, whatever
// order the counts were taken in.
//
// fork and release are one cluster of eight blocks each: the first half reads everything that the second
// half may overwrite, with the cluster's barrier between.  Bounded by latency: 256 forks of 32 parents 8.4 us, the
// release of 256 requests out of a pool of 18,000 pages 10.3 us, of a few 6.3 and 6.7 (with cold caches).
// copy: a block per page, head and tensor; 256 pages of 32 tokens x 8 heads x (128 + 128) channels 7.5 us, 4.5 TB/s
// there and 4.5 back.
#include <cooperative_groups.h>

#include "cache.h"
#include "common.cuh"

namespace cg = cooperative_groups;

namespace bpa {
namespace {

constexpr int kThreads = 1024, kCtas = 8, kAll = kThreads * kCtas;

// Exclusive running sum over the block in 32 bits; s [33]: the last word holds the block's total.
BPA_DEV int block_sum_before(int* s, int v) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();                       // s may still be read from the call before
    if (lane == 31) s[w] = x;
    __syncthreads();
    if (w == 0) {
        const int own = s[lane];
        int t = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t += y;
        }
        s[lane] = t - own;
        if (lane == 31) s[32] = t;
    }
    __syncthreads();
    return s[w] + x - v;
}

BPA_DEV void begin_status(uint32_t* status, bool bad, uint32_t where) {
    status[0] = bad ? ST_CHECK : 0u;
    status[1] = bad ? where : 0u;
    __threadfence();
}

__global__ void __launch_bounds__(kThreads) k_cache_fork(const ForkArgs a) {
    extern __shared__ int sm[];
    int* s_child = sm;                     // [R] the child that goes into the row; -1: none, -2: several
    int* s_len = s_child + a.R;            // [N] tokens of the parent; -1: not granted
    int* s_page = s_len + a.N;             // [N] place in the free list of the child's own page; -1: none
    __shared__ int s_sum[33], s_taken, s_bad;
    const auto cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank()), g = rank * kThreads + threadIdx.x;
    wait_for_previous();
    for (int r = threadIdx.x; r < a.R; r += kThreads) s_child[r] = -1;
    if (threadIdx.x == 0) s_taken = s_bad = 0;
    const int raw = *a.free_count, count = min(max(raw, 0), a.num_pages);
    __syncthreads();
    if (raw != count) s_bad = 1;
    for (int i = threadIdx.x; i < a.N; i += kThreads) {
        const int d = a.dst[i];
        if (d >= 0 && d < a.R && atomicCAS(s_child + d, -1, i) != -1) atomicExch(s_child + d, -2);
    }
    __syncthreads();
    int before = 0;
    for (int base = 0; base < a.N; base += kThreads) {
        const int i = base + threadIdx.x;
        int len = -1, need = 0;
        if (i < a.N) {
            const int s = a.src[i], d = a.dst[i];
            if (s >= 0 && s < a.R && d >= 0 && d < a.R && s_child[s] == -1 && s_child[d] == i && a.ctx[d] == 0) {
                len = a.ctx[s];
                if (len < 0 || len > static_cast<int64_t>(a.max_pages) * a.P) len = -1;
            }
            if (len < 0) s_bad = 1;
            else need = len % a.P != 0;
        }
        const int off = before + block_sum_before(s_sum, need);
        before += s_sum[32];
        if (i < a.N) {
            const bool ok = len >= 0 && (!need || off < count);
            s_len[i] = ok ? len : -1;
            s_page[i] = ok && need ? count - 1 - off : -1;
            if (ok && need) atomicMax(&s_taken, off + 1);
        }
    }
    __syncthreads();
    if (rank == 0 && threadIdx.x == 0) begin_status(a.status, s_bad, 0xCB8);
    cluster.sync();                        // every read of ctx_lens and free_count is done

    if (g == 0) *a.count_out = count - s_taken;
    for (int r = g; r < a.R; r += kAll) {
        const int i = s_child[r], len = i >= 0 ? s_len[i] : -1;
        if (len >= 0) a.ctx_out[r] = len;
        else if (a.ctx_out != a.ctx) a.ctx_out[r] = a.ctx[r];
    }
    const int lane = threadIdx.x & 31;
    for (int i = g >> 5; i < a.N; i += kAll / 32) {      // a warp to a child
        const int len = s_len[i], full = len < 0 ? 0 : len / a.P;
        const int32_t* from = a.table + static_cast<int64_t>(len < 0 ? 0 : a.src[i]) * a.max_pages;
        int32_t* to = a.table + static_cast<int64_t>(len < 0 ? 0 : a.dst[i]) * a.max_pages;
        for (int j = lane; j < full; j += 32) {
            const int id = from[j];
            const bool there = id >= 0 && id < a.num_pages;
            if (there) atomicAdd(a.refs + id, 1);
            else report(a.status, ST_CHECK, 0xCB9);
            to[j] = there ? id : -1;
        }
        if (lane) continue;
        int src = -1, dst = -1;
        if (s_page[i] >= 0) {
            src = from[full];
            dst = a.free_pages[s_page[i]];
            if (dst < 0 || dst >= a.num_pages) dst = -1;
            to[full] = dst;
            if (src < 0 || src >= a.num_pages || dst < 0) {
                report(a.status, ST_CHECK, 0xCB9);
                src = dst = -1;
            }
        }
        a.copy_src[i] = src;
        a.copy_dst[i] = dst;
    }
}

__global__ void __launch_bounds__(kThreads) k_cache_release(const ReleaseArgs a) {
    __shared__ int s_keep[kPlanMaxR / kCtas + 1];        // of the requests of this block: tokens that stay; -1: all
    __shared__ int s_gone[kThreads / 32], s_all[kCtas];
    const auto cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank()), lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    wait_for_previous();
    const int raw = *a.free_count, count = min(max(raw, 0), a.num_pages);
    if (rank == 0 && threadIdx.x == 0) begin_status(a.status, raw != count, 0xCB8);
    // this block's requests: rank, rank + kCtas, ..
    bool bad = false;
    for (int x = threadIdx.x; x * kCtas + rank < a.R; x += kThreads) {
        const int r = x * kCtas + rank, ctx = a.ctx[r], keep = a.keep[r];
        bool ok = keep >= 0 && keep <= ctx && ctx <= static_cast<int64_t>(a.max_pages) * a.P;
        if (ok && keep < ctx && keep % a.P) {            // the page that the request ends in must be its own
            const int id = a.table[static_cast<int64_t>(r) * a.max_pages + keep / a.P];
            ok = id >= 0 && id < a.num_pages && a.refs[id] == 0;
        }
        s_keep[x] = ok ? keep : -1;
        bad |= !ok;
    }
    cluster.sync();                        // every read of the counts is done, the status word is clear
    if (bad) report(a.status, ST_CHECK, 0xCBA);
    for (int x = warp; x * kCtas + rank < a.R; x += kThreads / 32) {
        const int r = x * kCtas + rank, ctx = a.ctx[r], keep = s_keep[x];
        if (keep < 0) continue;
        for (int j = (keep + a.P - 1) / a.P + lane; j < (ctx + a.P - 1) / a.P; j += 32) {
            const int id = a.table[static_cast<int64_t>(r) * a.max_pages + j];
            if (id >= 0 && id < a.num_pages) atomicSub(a.refs + id, 1);
            else report(a.status, ST_CHECK, 0xCB9);
        }
    }
    __threadfence();
    cluster.sync();                        // every holder has been taken
    for (int x = threadIdx.x; x * kCtas + rank < a.R; x += kThreads) {
        const int r = x * kCtas + rank;
        if (s_keep[x] >= 0) a.ctx_out[r] = s_keep[x];
        else if (a.ctx_out != a.ctx) a.ctx_out[r] = a.ctx[r];
    }
    // pages without a holder, in order: a warp takes a stretch of ids, 32 at a time
    const int per = (a.num_pages + kCtas * 32 - 1) / (kCtas * 32), stretch = (per + 31) / 32 * 32;
    const int64_t first = (static_cast<int64_t>(rank) * 32 + warp) * stretch;
    const int last = static_cast<int>(min(first + stretch, static_cast<int64_t>(a.num_pages)));
    int mine = 0;
#pragma unroll 4
    for (int64_t b = first; b < last; b += 32) {
        const int v = b + lane < last ? __ldcg(a.refs + b + lane) : 0;
        mine += __popc(__ballot_sync(0xffffffffu, v < 0));
    }
    if (lane == 0) s_gone[warp] = mine;
    __syncthreads();
    if (threadIdx.x == 0) {
        int t = 0;
        for (int w = 0; w < kThreads / 32; ++w) {
            const int n = s_gone[w];
            s_gone[w] = t;
            t += n;
        }
        for (int c = 0; c < kCtas; ++c) cluster.map_shared_rank(s_all, c)[rank] = t;
    }
    cluster.sync();
    int at = count + s_gone[warp];
    for (int c = 0; c < rank; ++c) at += s_all[c];
    for (int64_t b = first; b < last && mine; b += 32) {
        const int id = static_cast<int>(b) + lane, v = b + lane < last ? __ldcg(a.refs + id) : 0;
        const unsigned gone = __ballot_sync(0xffffffffu, v < 0);
        if (v < 0) {
            if (v < -1) report(a.status, ST_CHECK, 0xCBB);         // given up more often than held
            const int place = at + __popc(gone & ((1u << lane) - 1));
            if (place < a.num_pages) a.free_pages[place] = id;
            else report(a.status, ST_CHECK, 0xCBB);
            a.refs[id] = 0;
        }
        at += __popc(gone);
    }
    if (rank == 0 && threadIdx.x == 0) {
        int t = count;
        for (int c = 0; c < kCtas; ++c) t += s_all[c];
        *a.count_out = min(t, a.num_pages);
    }
}

constexpr int kCopyThreads = 128;

template <typename V>
__global__ void __launch_bounds__(kCopyThreads) k_cache_copy(const CopyArgs a) {
    wait_for_previous();
    if (blockIdx.x == gridDim.x - 1) {     // looks the pairs over for the status word, so that nothing clears it before
        __shared__ int s_bad;
        if (threadIdx.x == 0) s_bad = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < a.N; i += kCopyThreads) {
            const int x = a.src[i], y = a.dst[i];
            const bool none = x == -1 && y == -1;
            if (!none && (x < 0 || x >= a.num_pages || y < 0 || y >= a.num_pages)) s_bad = 1;
        }
        __syncthreads();
        if (threadIdx.x < 2) a.status[threadIdx.x] = !s_bad ? 0u : threadIdx.x ? 0xCBCu : static_cast<uint32_t>(ST_CHECK);
        return;
    }
    const int i = blockIdx.x / (2 * a.Hkv), hw = blockIdx.x - i * 2 * a.Hkv, h = hw >> 1;
    const bool is_v = hw & 1;
    const int64_t x = a.src[i], y = a.dst[i];
    if (x < 0 || x >= a.num_pages || y < 0 || y >= a.num_pages || x == y) return;
    const int64_t ps = is_v ? a.vcs[0] : a.kcs[0], hs = is_v ? a.vcs[1] : a.kcs[1], ts = is_v ? a.vcs[2] : a.kcs[2];
    uint8_t* base = (is_v ? a.vc : a.kc) + h * hs;
    float* scale = (is_v ? a.vscale : a.kscale) + h;
    if (threadIdx.x == 0) scale[y * a.Hkv] = scale[x * a.Hkv];
    const int units = (is_v ? a.dv : a.d) / static_cast<int>(sizeof(V)), n = units * a.P;
    const uint8_t* from = base + x * ps;
    uint8_t* to = base + y * ps;
#pragma unroll 4
    for (int k = threadIdx.x; k < n; k += kCopyThreads) {
        const int t = k / units;
        const int64_t at = t * ts + static_cast<int64_t>(k - t * units) * static_cast<int>(sizeof(V));
        *reinterpret_cast<V*>(to + at) = *reinterpret_cast<const V*>(from + at);
    }
}

template <typename... P, typename... A>
cudaError_t launch_cluster(size_t smem, cudaStream_t s, void (*kernel)(P...), A... args) {
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = kCtas;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCtas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
}

}  // namespace

cudaError_t launch_cache_fork(const ForkArgs& a, cudaStream_t s) {
    const size_t smem = sizeof(int) * (static_cast<size_t>(a.R) + 2 * static_cast<size_t>(a.N));
    if (smem > 47 * 1024) {                // with the static part more than the 48 KB that need no asking
        const cudaError_t e = cudaFuncSetAttribute(k_cache_fork, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(sizeof(int) * 3 * kPlanMaxR));
        if (e != cudaSuccess) return e;
    }
    return launch_cluster(smem, s, k_cache_fork, a);
}

cudaError_t launch_cache_release(const ReleaseArgs& a, cudaStream_t s) { return launch_cluster(0, s, k_cache_release, a); }

cudaError_t launch_cache_copy(const CopyArgs& a, cudaStream_t s) {
    uintptr_t all = reinterpret_cast<uintptr_t>(a.kc) | reinterpret_cast<uintptr_t>(a.vc) | a.d | a.dv;
    for (int i = 0; i < 3; ++i) all |= static_cast<uintptr_t>(a.kcs[i]) | static_cast<uintptr_t>(a.vcs[i]);
    const dim3 grid(static_cast<unsigned>(static_cast<int64_t>(a.N) * 2 * a.Hkv + 1));
    return launch_early(grid, dim3(kCopyThreads), 0, s, all % 16 == 0 ? k_cache_copy<uint4> : k_cache_copy<uint8_t>, a);
}

}  // namespace bpa
