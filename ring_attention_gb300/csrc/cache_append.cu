// cache_append.cu - new keys and values into the pages of the 8-bit cache.
//
// A run is a stretch of rows with consecutive slots in one page.  For each run, head and tensor
// (k or v): s_new = the smallest power of two with amax <= 448 s_new, scale = max(old, s_new) (s_new
// alone where the run opens the page), the rows that the page already holds are moved to the new
// scale if it grew, and the run's rows are rounded to e4m3 once.  Powers of two make a move exact
// except below e4m3's smallest normal number (2^-6 of the new scale), where it rounds again: at most
// 2^-10 of the scale, half of e4m3's smallest step, per doubling.
#include "cache.h"
#include "common.cuh"
#include "e4m3.cuh"

namespace bpa {
namespace {

// VE consecutive channels of a row as float32 bit patterns (16 bytes at a time, or one element)
template <int VE>
BPA_DEV void load_row(const float* p, uint32_t (&v)[VE]) {
    if constexpr (VE == 1) {
        v[0] = __float_as_uint(__ldg(p));
    } else {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(p));
        v[0] = x.x;
        v[1] = x.y;
        v[2] = x.z;
        v[3] = x.w;
    }
}
template <int VE>
BPA_DEV void load_row(const __nv_bfloat16* p, uint32_t (&v)[VE]) {
    if constexpr (VE == 1) {
        v[0] = static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(p))) << 16;
    } else {
        const uint4 x = __ldg(reinterpret_cast<const uint4*>(p));
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = w[i] << 16;
            v[2 * i + 1] = w[i] & 0xffff0000u;
        }
    }
}

// The smallest power of two s >= 2^-100 with amax <= 448 s = 1.75 * 2^8 s; 0 for amax = 0.  From the
// bits: amax = 1.f * 2^e gives s = 2^(e - 8) where 1.f <= 1.75 and 2^(e - 7) above.
BPA_DEV float scale_for(float amax) {
    if (!(amax > 0.f)) return 0.f;
    const uint32_t u = __float_as_uint(amax);
    const int e = static_cast<int>(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float(static_cast<uint32_t>(max(e, 27)) << 23);   // 27 - 127 = -100
}

// One warp per (ROWS rows, head, tensor): it takes the runs that begin in its rows, one after the
// other, reading a run twice (largest magnitude, then codes; the second time from L2).  Bounded by the
// latency of a warp's chain (slots, rows, scale, rows again) rather than by bytes: prompts of 19,000
// rows x 8 heads x (128 + 64) bf16 channels take 31 us, 2.9 TB/s of their 90 MB; loops over rows are
// unrolled sixteen times (four: 33 us), though a thread's 64 registers do not hold sixteen loads at once.
// ROWS = 1 when requests bring few rows (every row is then a run of its own, or nearly); ROWS = 16 for
// prompts, whose runs are whole pages: sixteen times fewer warps that find no beginning.  The last block
// looks the slots over for the status word, so that nothing has to clear it before; as it starts late,
// that is 0.7 of the 31 us, and 11 of the 95 that four times the rows take.  ONE: a row takes no more than
// 32 lanes, so the loops over rows are the only ones and their loads overlap (with a loop over a row's
// units inside: 41 us).
template <typename E, int VE, int ROWS, bool ONE>
__global__ void __launch_bounds__(128) k_cache_append(const AppendArgs a) {
    wait_for_previous();
    const int lane = threadIdx.x & 31, cap = a.P * a.num_pages;
    if (blockIdx.x == gridDim.x - 1) {
        __shared__ int s_bad;
        if (threadIdx.x == 0) s_bad = 0;
        __syncthreads();
        for (int t = threadIdx.x; t < a.T; t += 128)
            if (static_cast<uint32_t>(a.slots[t]) + 1u > static_cast<uint32_t>(cap)) s_bad = 1;   // outside [-1, cap)
        __syncthreads();
        if (threadIdx.x < 2) a.status[threadIdx.x] = !s_bad ? 0u : threadIdx.x ? 0xCB0u : static_cast<uint32_t>(ST_CHECK);
        return;
    }
    const int64_t item = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    const int first = static_cast<int>(item / (2 * a.Hkv)) * ROWS;
    if (first >= a.T) return;
    const int hw = static_cast<int>(item % (2 * a.Hkv)), h = hw >> 1;
    const bool is_v = hw & 1;
    const int c = is_v ? a.dv : a.d;
    const int64_t xs = is_v ? a.vs[0] : a.ks[0], ts = is_v ? a.vcs[2] : a.kcs[2];
    const E* rows = static_cast<const E*>(is_v ? a.v : a.k) + h * (is_v ? a.vs[1] : a.ks[1]);
    const int units = c / VE, across = min(units, 32);             // lanes of a row
    const int down = 32 / across, li = lane / across, lu = lane % across;
    const bool active = li < down;

    // lane i: slot of row first + i and of the one before
    const int mine = lane < ROWS && first + lane < a.T ? a.slots[first + lane] : -1;
    const int before = lane < ROWS && first + lane > 0 && first + lane < a.T ? a.slots[first + lane - 1] : -1;
    unsigned begins = __ballot_sync(0xffffffffu, mine >= 0 && mine < cap && (mine % a.P == 0 || before != mine - 1));
    while (begins) {
        const int b = __ffs(begins) - 1;
        begins &= begins - 1;
        const int t0 = first + b, slot = __shfl_sync(0xffffffffu, mine, b);
        const int page = slot / a.P, off = slot - page * a.P;
        float* scale = (is_v ? a.vscale : a.kscale) + static_cast<int64_t>(page) * a.Hkv + h;
        const float old = off ? *scale : 0.f;
        int n = 1;                                                 // rows of the run
        while (off + n < a.P) {
            const int i = n + lane, t = t0 + i;
            const unsigned more = __ballot_sync(0xffffffffu, t < a.T && off + i < a.P && a.slots[min(t, a.T - 1)] == slot + i);
            n += more == 0xffffffffu ? 32 : __ffs(~more) - 1;
            if (more != 0xffffffffu) break;
        }
        const E* x = rows + t0 * xs;
        // the largest magnitude as bits: at and above 0x7f800000 infinities and NaN are among the rows
        uint32_t top = 0;
        if (active) {
#pragma unroll 16
            for (int i = li; i < n; i += down)
                for (int u = lu; ONE ? u == lu : u < units; u += across) {
                    uint32_t v[VE];
                    load_row<VE>(x + i * xs + u * VE, v);
#pragma unroll
                    for (int e = 0; e < VE; ++e) top = max(top, v[e] & 0x7fffffffu);
                }
        }
        top = __reduce_max_sync(0xffffffffu, top);
        const bool plain = top < 0x7f800000u;
        if (!plain) {
            top = 0;
            if (active)
                for (int i = li; i < n; i += down)
                    for (int u = lu; ONE ? u == lu : u < units; u += across) {
                        uint32_t v[VE];
                        load_row<VE>(x + i * xs + u * VE, v);
#pragma unroll
                        for (int e = 0; e < VE; ++e)
                            if ((v[e] & 0x7fffffffu) < 0x7f800000u) top = max(top, v[e] & 0x7fffffffu);
                    }
            top = __reduce_max_sync(0xffffffffu, top);
        }
        const float s = fmaxf(old, scale_for(__uint_as_float(top)));
        uint8_t* out = is_v ? a.vc + page * a.vcs[0] + h * a.vcs[1] : a.kc + page * a.kcs[0] + h * a.kcs[1];
        if (off && s > old) {
            const float ratio = old / s;
            if (active)
#pragma unroll 2
                for (int i = li; i < off; i += down)
                    for (int u = lu; ONE ? u == lu : u < units; u += across) {
                        uint8_t* p = out + i * ts + u * VE;
                        if constexpr (VE == 1) {
                            *p = static_cast<uint8_t>(e4m3_pair(from_e4m3(*p) * ratio, 0.f));
                        } else {
                            uint32_t* q = reinterpret_cast<uint32_t*>(p);
#pragma unroll
                            for (int k = 0; k < VE / 4; ++k) q[k] = rescaled4(q[k], ratio);
                        }
                    }
        }
        const float inv = s > 0.f ? 1.f / s : 1.f;
        out += off * ts;
        if (active) {
#pragma unroll 16
            for (int i = li; i < n; i += down)
                for (int u = lu; ONE ? u == lu : u < units; u += across) {
                    uint32_t v[VE];
                    load_row<VE>(x + i * xs + u * VE, v);
                    if (!plain)
#pragma unroll
                        for (int e = 0; e < VE; ++e)               // an infinity is stored as NaN
                            if ((v[e] & 0x7fffffffu) == 0x7f800000u) v[e] = 0x7fc00000u;
                    uint8_t* p = out + i * ts + u * VE;
                    if constexpr (VE == 1) {
                        *p = static_cast<uint8_t>(e4m3_pair(__uint_as_float(v[0]) * inv, 0.f));
                    } else {
                        uint32_t w[VE / 4];
#pragma unroll
                        for (int k = 0; k < VE / 4; ++k)
                            w[k] = e4m3_pair(__uint_as_float(v[4 * k]) * inv, __uint_as_float(v[4 * k + 1]) * inv) |
                                   e4m3_pair(__uint_as_float(v[4 * k + 2]) * inv, __uint_as_float(v[4 * k + 3]) * inv) << 16;
                        if constexpr (VE == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
                        else *reinterpret_cast<uint32_t*>(p) = w[0];
                    }
                }
        }
        __syncwarp();
        if (lane == 0) *scale = s;
        __syncwarp();
    }
}

template <typename E, int VE>
cudaError_t launch(const AppendArgs& a, cudaStream_t s) {
    // Measured both ways: 128 single rows x 8 heads 2.9 us a row to a warp, 16 us sixteen to one; the prompts
    // above 94 and 31 us.  Unknown: by the rows in all.
    const bool one = (a.d > a.dv ? a.d : a.dv) <= 32 * VE, few = a.max_new > 0 ? a.max_new <= 8 : a.T <= 512;
    const int rows = few ? 1 : 16;
    const int64_t items = static_cast<int64_t>((a.T + rows - 1) / rows) * 2 * a.Hkv;
    const dim3 grid(static_cast<unsigned>((items + 3) / 4 + 1));
    auto kernel = few ? (one ? k_cache_append<E, VE, 1, true> : k_cache_append<E, VE, 1, false>)
                      : (one ? k_cache_append<E, VE, 16, true> : k_cache_append<E, VE, 16, false>);
    return launch_early(grid, dim3(128), 0, s, kernel, a);
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs& a, cudaStream_t s) {
    // 16-byte loads and 8- or 4-byte stores where everything is aligned to them
    const int ve = a.dtype == BPA_BF16 ? 8 : 4;
    const uintptr_t in = reinterpret_cast<uintptr_t>(a.k) | reinterpret_cast<uintptr_t>(a.v);
    uintptr_t out = reinterpret_cast<uintptr_t>(a.kc) | reinterpret_cast<uintptr_t>(a.vc) | a.d | a.dv;
    int64_t strides = 0;
    for (int i = 0; i < 2; ++i) strides |= a.ks[i] | a.vs[i];
    for (int i = 0; i < 3; ++i) out |= static_cast<uintptr_t>(a.kcs[i]) | static_cast<uintptr_t>(a.vcs[i]);
    const bool wide = in % 16 == 0 && strides % ve == 0 && out % ve == 0;
    if (a.dtype == BPA_BF16) return wide ? launch<__nv_bfloat16, 8>(a, s) : launch<__nv_bfloat16, 1>(a, s);
    return wide ? launch<float, 4>(a, s) : launch<float, 1>(a, s);
}

}  // namespace bpa
