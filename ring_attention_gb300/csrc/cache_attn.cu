// cache_attn.cu - attention over the paged 8-bit cache, any shape (CUDA cores, float32).
//
// One CTA per packed row and q head.  Its four warps take every fourth chunk of 32 keys: a lane per
// key for the scores (the row of q in shared memory), then a lane per channel for p V, with a running
// (max, denominator, numerator) of the warp; the four are merged at the end.
//
// Takes what the other kernels do not: head dims that are no multiple of 16 or above 256, pages other
// than 16, 32 or a multiple of 64 tokens, strides or bases that TMA does not take, more than 2^30 rows of
// a kv head in all.  Bounded by its instructions (every q head reads and decodes the codes of its kv head
// again): 8 requests of 1,000 tokens with 8 heads over 2 of 72 channels 94 us, of 512 channels 383 us; 64
// requests of 8,192 tokens, 32 heads over 8 of 128 channels, pages of 50 tokens 8.6 ms where pages of 64
// let the matrix instructions take 0.155 ms.
#include <cuda_fp8.h>

#include "cache.h"
#include "common.cuh"

namespace bpa {
namespace {

constexpr int kWarps = 4, kMaxD = 512;

BPA_DEV float dec(uint8_t c) { return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3))); }
BPA_DEV float load_f32(const float* p) { return __ldg(p); }
BPA_DEV float load_f32(const __nv_bfloat16* p) { return __bfloat162float(*p); }
BPA_DEV void store_f32(float* p, float x) { *p = x; }
BPA_DEV void store_f32(__nv_bfloat16* p, float x) { *p = __float2bfloat16(x); }

template <typename E>
__global__ void __launch_bounds__(kWarps * 32) k_cache_attn_simt(const CacheAttnArgs a) {
    __shared__ float s_q[kMaxD], s_acc[kWarps][kMaxD], s_m[kWarps], s_l[kWarps];
    const int t = blockIdx.x, h = blockIdx.y, hk = h / a.G;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (t < __ldg(a.cu_q) || t >= __ldg(a.cu_q + a.R)) return;
    int lo = 0, hi = a.R;                 // the request: the last whose first row is <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(a.cu_q + mid) <= t) lo = mid;
        else hi = mid;
    }
    const int r = lo;
    const Req rq = request_of(a, r);
    if (rq.bad && threadIdx.x == 0) report(a.status, ST_CHECK, 0xCC1);
    int k0, k1;
    row_keys(a, rq, t - rq.row0, k0, k1);
    const E* q = static_cast<const E*>(a.q) + t * a.qs[0] + h * a.qs[1];
    for (int j = threadIdx.x; j < a.d; j += kWarps * 32) s_q[j] = load_f32(q + j);
    __syncthreads();
    const int32_t* table = a.table + static_cast<int64_t>(r) * a.max_pages;
    float m = -INFINITY, l = 0.f, acc[kMaxD / 32];
#pragma unroll
    for (int j = 0; j < kMaxD / 32; ++j) acc[j] = 0.f;
    for (int64_t base = static_cast<int64_t>(k0) + 32 * warp; base <= k1; base += 32 * kWarps) {
        const int key = static_cast<int>(base) + lane;
        float z = -INFINITY, vscale = 0.f;
        int64_t at = -1;                  // the key's row of v, -1: none
        if (key <= k1) {
            const int pg = key / a.P, off = key - pg * a.P, id = __ldg(table + pg);
            if (id >= 0 && id < a.num_pages) {
                const uint8_t* k = a.kc + id * a.kcs[0] + hk * a.kcs[1] + off * a.kcs[2];
                float x = 0.f;
                for (int j = 0; j < a.d; ++j) x = fmaf(s_q[j], dec(__ldg(k + j)), x);
                z = x * __ldg(a.kscale + static_cast<int64_t>(id) * a.Hkv + hk) * a.scale;
                vscale = __ldg(a.vscale + static_cast<int64_t>(id) * a.Hkv + hk);
                at = id * a.vcs[0] + hk * a.vcs[1] + off * a.vcs[2];
            } else {
                report(a.status, ST_CHECK, 0xCC0);
            }
        }
        float mx = z;
#pragma unroll
        for (int o = 16; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        const float mn = fmaxf(m, mx);
        if (mn == -INFINITY && !__any_sync(0xffffffffu, z != z)) continue;   // nothing that counts so far
        const float ref = mn == -INFINITY ? 0.f : mn, fix = m == -INFINITY ? 0.f : expf(m - ref);
        const float p = at < 0 ? 0.f : expf(z - ref);
        float sum = p;
#pragma unroll
        for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        l = l * fix + sum;
        m = mn;
        const float w = p * vscale;
#pragma unroll
        for (int j = 0; j < kMaxD / 32; ++j) acc[j] *= fix;
        for (int i = 0; i < 32; ++i) {
            const int64_t ai = __shfl_sync(0xffffffffu, at, i);
            const float wi = __shfl_sync(0xffffffffu, w, i);
            if (ai < 0) continue;
#pragma unroll
            for (int j = 0; j < kMaxD / 32; ++j)
                if (j * 32 + lane < a.dv) acc[j] = fmaf(wi, dec(__ldg(a.vc + ai + j * 32 + lane)), acc[j]);
        }
    }
    if (lane == 0) {
        s_m[warp] = m;
        s_l[warp] = l;
    }
#pragma unroll
    for (int j = 0; j < kMaxD / 32; ++j) s_acc[warp][j * 32 + lane] = acc[j];
    __syncthreads();
    float mt = -INFINITY;
    for (int w = 0; w < kWarps; ++w) mt = fmaxf(mt, s_m[w]);
    const float sink = a.sink ? __ldg(a.sink + h) : -INFINITY;
    mt = fmaxf(mt, sink);
    const float ref = mt == -INFINITY ? 0.f : mt;
    float f[kWarps], lt = a.sink ? expf(sink - ref) : 0.f;
    for (int w = 0; w < kWarps; ++w) {
        f[w] = expf(s_m[w] - ref);
        lt += s_l[w] * (s_l[w] == 0.f ? 0.f : f[w]);
    }
    const float inv = lt == 0.f ? 0.f : 1.f / lt;
    E* o = static_cast<E*>(a.o) + t * a.os[0] + h * a.os[1];
    for (int j = threadIdx.x; j < a.dv; j += kWarps * 32) {
        float x = 0.f;
        for (int w = 0; w < kWarps; ++w) x += s_l[w] == 0.f ? 0.f : s_acc[w][j] * f[w];
        store_f32(o + j, x * inv);
    }
    if (a.m && threadIdx.x == 0) {
        a.m[static_cast<int64_t>(h) * a.T + t] = mt;
        a.l[static_cast<int64_t>(h) * a.T + t] = lt;
    }
}

}  // namespace

cudaError_t launch_cache_attn_simt(const CacheAttnArgs& a, cudaStream_t s) {
    const dim3 grid(a.T, a.Hq);
    if (a.dtype == BPA_BF16) k_cache_attn_simt<__nv_bfloat16><<<grid, kWarps * 32, 0, s>>>(a);
    else k_cache_attn_simt<float><<<grid, kWarps * 32, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace bpa
