// cache_plan.cu - block tables and slot maps of one serving step, built on the device.
//
// With have = ceil(ctx / P), need = ceil((ctx + new) / P) - have and upto = the running sum of
// need, request r's j-th new page is free_pages[count - 1 - (upto_r - need_r) - j], and it is
// granted when it needs none or upto_r <= count.  The two running sums (of rows and of pages)
// are block scans; the rest is one thread per row of the packed buffers and per taken page, which
// find their request by a binary search over the sums in shared memory.
//
// Bounded by latency: a step of 256 generating requests moves 7 KB, so its time is the launch, one
// round trip for the lengths, the scans and one dependent round trip for the page ids: 5.3 us.  A
// cluster of eight CTAs shares the rows (each repeats the scans, which cost less than handing the
// sums over): 64 requests of 64,000 rows in all 11.1 us against 53.8 with one CTA, 4,096 rows 5.5 against
// 8.6, and one row for each of 256 requests 5.3 against 5.3, so that no size wants fewer.  The cluster
// barrier between the last read of the lengths and the first write is what lets ctx_lens_out and
// free_count_out overwrite their inputs.
#include <cooperative_groups.h>

#include "cache.h"
#include "common.cuh"

namespace cg = cooperative_groups;

namespace bpa {
namespace {

constexpr int kThreads = 1024;
constexpr int kCtas = 8;                // of the cluster (the largest that needs no opt-in)

struct Scan {
    long long warp[kThreads / 32];
    long long carry;
};
static_assert(2 * sizeof(Scan) + 64 <= 1024, "the kernel's static shared memory");   // launch_cache_plan counts on it

// Exclusive running sum of v over the block, continued from s.carry, which moves on by the total.
__device__ long long block_scan(Scan& s, long long v) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    long long x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s.warp[w] = x;
    __syncthreads();
    if (w == 0) {
        long long t = s.warp[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, t, o);
            if (lane >= o) t += y;
        }
        s.warp[lane] = t;
    }
    __syncthreads();
    const long long before = s.carry + (w ? s.warp[w - 1] : 0);
    const long long total = s.warp[kThreads / 32 - 1];
    __syncthreads();
    if (threadIdx.x == 0) s.carry += total;
    __syncthreads();
    return before + x - v;
}

// The last of the n ascending values that is <= x (values[0] <= x).
__device__ __forceinline__ int last_not_above(const int* values, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (values[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads) k_cache_plan(const PlanArgs a) {
    extern __shared__ int sm[];
    int* s_cu = sm;                       // [R + 1] first row of each request, clamped to T
    int* s_off = s_cu + a.R + 1;          // [R] pages taken before the request
    int* s_ctx = s_off + a.R;             // [R] tokens in the cache; the top bit: the request waits
    __shared__ Scan rows, pages;
    __shared__ int s_taken, s_bad;
    const auto cluster = cg::this_cluster();
    const int rank = static_cast<int>(cluster.block_rank()), ranks = static_cast<int>(cluster.num_blocks());
    if (threadIdx.x == 0) {
        rows.carry = pages.carry = 0;
        s_taken = 0;
        s_bad = 0;
    }
    wait_for_previous();
    const int raw = *(a.free_count), count = min(max(raw, 0), a.num_pages);
    __syncthreads();
    if (raw != count) s_bad = 1;
    for (int base = 0; base < a.R; base += kThreads) {
        const int r = base + threadIdx.x;
        const int ctx = r < a.R ? *(a.ctx + r) : 0, add = r < a.R ? *(a.add + r) : 0;
        const int n = max(add, 0);
        const long long row = block_scan(rows, n), last = static_cast<long long>(ctx) + n;
        const bool bad = ctx < 0 || add < 0 || last > static_cast<long long>(a.max_pages) * a.P || row + n > a.T;
        const int need = bad ? 0 : static_cast<int>((last + a.P - 1) / a.P) - (ctx + a.P - 1) / a.P;
        const long long off = block_scan(pages, need);
        if (r < a.R) {
            const bool ok = !bad && (need == 0 || off + need <= count);
            s_cu[r] = static_cast<int>(min(row, static_cast<long long>(a.T)));
            // clamped where no page is taken any more (the sum is then above every page index)
            s_off[r] = static_cast<int>(min(off, static_cast<long long>(INT_MAX)));
            s_ctx[r] = (ctx & INT_MAX) | (ok ? 0 : INT_MIN);
            if (ok && need) atomicMax(&s_taken, static_cast<int>(off) + need);
            if (bad) s_bad = 1;
        }
    }
    __syncthreads();                      // every thread has said whether its requests are bad
    if (threadIdx.x == 0) {
        s_cu[a.R] = static_cast<int>(min(rows.carry, static_cast<long long>(a.T)));
        if (rank == 0) {                  // cleared before the barrier, so before any later report
            a.status[0] = s_bad ? ST_CHECK : 0u;
            a.status[1] = s_bad ? 0xCA0u : 0u;
            __threadfence();
        }
    }
    cluster.sync();                       // every read of ctx_lens and free_count is done

    const int g = rank * kThreads + threadIdx.x, step = ranks * kThreads;
    const int taken = s_taken, total = s_cu[a.R];
    if (g == 0) *a.count_out = count - taken;
    for (int r = g; r <= a.R; r += step) {
        a.cu_q[r] = s_cu[r];
        if (r == a.R) break;
        const int c = s_ctx[r];
        // rows cut off at T belong to requests that wait, so the clamped sums are exact for the others
        const int sum = (c & INT_MAX) + (s_cu[r + 1] - s_cu[r]);
        a.kv_lens[r] = c < 0 ? 0 : sum;
        if (c >= 0) a.ctx_out[r] = sum;
        else if (a.ctx_out != a.ctx) a.ctx_out[r] = *(a.ctx + r);
    }
    for (int n = g; n < taken; n += step) {
        const int r = last_not_above(s_off, a.R, n);
        int id = *(a.free_pages + count - 1 - n);
        if (id < 0 || id >= a.num_pages) {
            report(a.status, ST_CHECK, 0xCA1);
            id = -1;
        }
        const int have = (s_ctx[r] & INT_MAX) / a.P + ((s_ctx[r] & INT_MAX) % a.P != 0);
        a.table[static_cast<int64_t>(r) * a.max_pages + have + (n - s_off[r])] = id;
    }
    for (int t = g; t < a.T; t += step) {
        int slot = -1, pos = -1;
        if (t < total) {
            const int r = last_not_above(s_cu, a.R, t);
            const int ctx = s_ctx[r];
            if (ctx >= 0) {
                pos = ctx + (t - s_cu[r]);
                const int j = pos / a.P, have = ctx / a.P + (ctx % a.P != 0);
                const int id = j < have ? *(a.table + static_cast<int64_t>(r) * a.max_pages + j)
                                        : *(a.free_pages + count - 1 - (s_off[r] + j - have));
                if (id >= 0 && id < a.num_pages) {
                    slot = id * a.P + (pos - j * a.P);
                } else {
                    report(a.status, ST_CHECK, 0xCA1);
                    pos = -1;
                }
            }
        }
        a.slots[t] = slot;
        if (a.positions) a.positions[t] = pos;
    }
}

}  // namespace

cudaError_t launch_cache_plan(const PlanArgs& a, cudaStream_t s) {
    const size_t smem = sizeof(int) * (3 * static_cast<size_t>(a.R) + 1);
    // a kernel has 48 KB without asking, its static part (the scans, below 1 KB) included
    if (smem > 47 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(k_cache_plan, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(sizeof(int) * (3 * kPlanMaxR + 1)));
        if (e != cudaSuccess) return e;
    }
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
    return cudaLaunchKernelEx(&cfg, k_cache_plan, a);
}

}  // namespace bpa
