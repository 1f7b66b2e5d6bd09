// cache_append.cu - new keys and values into the pages of the 8-bit cache.
//
// A run is a stretch of rows with consecutive slots in one page.  For each run, head and tensor
// (k or v): s_new = the smallest power of two with amax <= 448 s_new, scale = max(old, s_new) (s_new
// alone where the run opens the page), the rows that the page already holds are moved to the new
// scale if it grew, and the run's rows are rounded to e4m3 once.  Powers of two make a move exact
// except below e4m3's smallest normal number (2^-6 of the new scale), where it rounds again: at most
// 2^-10 of the scale, half of e4m3's smallest step, per doubling.
#include <cuda_fp8.h>

#include "cache.h"
#include "common.cuh"

namespace bpa {
namespace {

BPA_DEV float load_f32(const float* p) { return __ldg(p); }
BPA_DEV float load_f32(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// round to nearest even; infinities (and what lies past 448, which the scale rules out) become NaN
BPA_DEV uint8_t to_e4m3(float x) {
    return fabsf(x) < INFINITY ? static_cast<uint8_t>(__nv_cvt_float_to_fp8(x, __NV_SATFINITE, __NV_E4M3)) : 0x7f;
}
BPA_DEV float from_e4m3(uint8_t c) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}

// The smallest power of two s >= 2^-100 with amax <= 448 s = 1.75 * 2^8 s; 0 for amax = 0.  From the
// bits: amax = 1.f * 2^e gives s = 2^(e - 8) where 1.f <= 1.75 and 2^(e - 7) above.
BPA_DEV float scale_for(float amax) {
    if (!(amax > 0.f)) return 0.f;
    const uint32_t u = __float_as_uint(amax);
    const int e = static_cast<int>(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float(static_cast<uint32_t>(max(e, 27)) << 23);   // 27 - 127 = -100
}

// One warp per (row, head, tensor): the warp of a run's first row takes the run.
template <typename E>
__global__ void __launch_bounds__(128) k_cache_append(const AppendArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int t0 = static_cast<int>(item / (2 * a.Hkv));
    if (t0 >= a.T) return;
    const int hw = static_cast<int>(item % (2 * a.Hkv)), h = hw >> 1;
    const bool is_v = hw & 1;
    const int slot = __ldg(a.slots + t0);
    if (slot < 0) return;
    const int cap = a.P * a.num_pages;
    if (slot >= cap) {
        if (lane == 0) report(a.status, ST_CHECK, 0xCB0);
        return;
    }
    const int page = slot / a.P, off = slot - page * a.P;
    if (off && t0 && __ldg(a.slots + t0 - 1) == slot - 1) return;   // not the run's first row
    int n = 1;                                                      // rows of the run
    for (;;) {
        const int i = n + lane, t = t0 + i;
        const bool in = t < a.T && off + i < a.P && __ldg(a.slots + t) == slot + i;
        const unsigned b = __ballot_sync(0xffffffffu, in);
        if (b != 0xffffffffu) {
            n += __ffs(~b) - 1;
            break;
        }
        n += 32;
    }
    const int c = is_v ? a.dv : a.d;
    const E* x = static_cast<const E*>(is_v ? a.v : a.k) + t0 * (is_v ? a.vs[0] : a.ks[0]) + h * (is_v ? a.vs[1] : a.ks[1]);
    const int64_t xs = is_v ? a.vs[0] : a.ks[0];
    const int64_t ts = is_v ? a.vcs[2] : a.kcs[2];
    uint8_t* out = is_v ? a.vc + page * a.vcs[0] + h * a.vcs[1] : a.kc + page * a.kcs[0] + h * a.kcs[1];
    float* scale = (is_v ? a.vscale : a.kscale) + static_cast<int64_t>(page) * a.Hkv + h;
    float amax = 0.f;
    for (int i = 0; i < n; ++i)
        for (int j = lane; j < c; j += 32) {
            const float y = fabsf(load_f32(x + i * xs + j));
            if (y < INFINITY) amax = fmaxf(amax, y);
        }
#pragma unroll
    for (int o = 16; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float old = off ? *scale : 0.f;
    const float s = fmaxf(old, scale_for(amax));
    if (s > old && off) {
        const float ratio = old / s;
        for (int i = 0; i < off; ++i)
            for (int j = lane; j < c; j += 32) out[i * ts + j] = to_e4m3(from_e4m3(out[i * ts + j]) * ratio);
    }
    const float inv = s > 0.f ? 1.f / s : 1.f;
    for (int i = 0; i < n; ++i)
        for (int j = lane; j < c; j += 32) out[(off + i) * ts + j] = to_e4m3(load_f32(x + i * xs + j) * inv);
    __syncwarp();
    if (lane == 0) *scale = s;
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t s) {
    const int64_t blocks = (static_cast<int64_t>(a.T) * 2 * a.Hkv + 3) / 4;
    if (a.dtype == BPA_BF16) k_cache_append<__nv_bfloat16><<<static_cast<unsigned>(blocks), 128, 0, s>>>(a);
    else k_cache_append<float><<<static_cast<unsigned>(blocks), 128, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace bpa
