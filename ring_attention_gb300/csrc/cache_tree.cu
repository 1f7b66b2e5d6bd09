// cache_tree.cu - masks and positions of drafted trees from their parents.
//
//   mask(i) = {i} and mask(parent(i));  position(i) = context + (number of i's ancestors among the drafts).
//   Under a window: of the ancestors those up to `wl` steps above i.
//
// A block per request: its parents in shared memory, a thread per row and word of a mask walks from the row
// to its root.  Bounded by latency (lengths, then parents, then a walk as deep as the tree): 32 trees of 8 to 64
// rows 4.0 us, one of 26 rows 3.7, and 1.5 for clearing the status word in front (a step pays both once, its
// layers share the masks).  Every word walks the whole path, so far larger trees are bounded by those steps, rows x
// words x depth of them: with the clearing, chains of 64 rows 6.2 us, of 256 rows 62, of 1,024 rows 3,360, a tree of
// 1,024 rows that branches 30 wide 311 (one request or 32).
#include "cache.h"
#include "common.cuh"

namespace bpa {
namespace {

constexpr int kThreads = 128;

__global__ void __launch_bounds__(kThreads) k_cache_tree(const TreeArgs a) {
    __shared__ int s_par[32 * kMaxTreeWords];
    const int r = blockIdx.x;
    wait_for_previous();
    const int row0 = min(max(a.cu_q[r], 0), a.T), n = max(min(a.cu_q[r + 1], a.T) - row0, 0), len = a.kv_lens[r];
    // a request that waits has no tokens; its rows see nothing
    const bool ok = n <= len && n <= 32 * a.words;
    if (!ok && len != 0 && threadIdx.x == 0) report(a.status, ST_CHECK, 0xCF0);
    if (ok) {
        for (int i = threadIdx.x; i < n; i += kThreads) {
            int p = a.parents[row0 + i];
            if (p < -1 || p >= i) {
                report(a.status, ST_CHECK, 0xCF1);
                p = -1;
            }
            s_par[i] = p;
        }
        __syncthreads();
    }
    for (int64_t x = threadIdx.x; x < static_cast<int64_t>(n) * a.words; x += kThreads) {
        const int i = static_cast<int>(x / a.words), w = static_cast<int>(x - static_cast<int64_t>(i) * a.words);
        uint32_t bits = 0;
        int above = -1;
        if (ok)
            for (int j = i; j >= 0; j = s_par[j]) {          // parents come first, so this ends
                ++above;
                if (j >> 5 == w && (a.wl < 0 || above <= a.wl)) bits |= 1u << (j & 31);
            }
        a.tree[static_cast<int64_t>(row0 + i) * a.words + w] = bits;
        if (w == 0 && a.positions) a.positions[row0 + i] = ok ? len - n + above : -1;
    }
    // rows of no request
    const int first = min(max(a.cu_q[0], 0), a.T), last = min(max(a.cu_q[a.R], 0), a.T);
    const int64_t out = static_cast<int64_t>(first) + a.T - last;
    for (int64_t x = static_cast<int64_t>(r) * kThreads + threadIdx.x; x < out; x += static_cast<int64_t>(a.R) * kThreads) {
        const int t = static_cast<int>(x < first ? x : last + x - first);
        for (int w = 0; w < a.words; ++w) a.tree[static_cast<int64_t>(t) * a.words + w] = 0;
        if (a.positions) a.positions[t] = -1;
    }
}

}  // namespace

cudaError_t launch_cache_tree(const TreeArgs& a, cudaStream_t s) {
    return launch_early(dim3(a.R), dim3(kThreads), 0, s, k_cache_tree, a);
}

}  // namespace bpa
