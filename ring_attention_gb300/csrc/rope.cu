// rope.cu - RMS norm of each head of q and k and the rotation by its token's position, and its gradients.
//
//   xh = x / sqrt(mean x^2 + eps),  n = w xh,  and for each pair (a, b) of n's first `rot` channels
//   a' = a cos t - b sin t,  b' = b cos t + a sin t  with t = position * inv_freq.
//   Backward: g = the gradient rotated by -t;  dw = sum g xh;  e = w g;  dx = r (e - xh mean(e xh)).
//
// The angle is the exact product of two numbers of 31 and 24 bits, taken in whole turns: inv_freq / 2 pi as a
// fraction of 64 bits (wrapping is what full turns do), times the position, so a far position loses
// nothing; the top 32 bits of the product, less the nearest quarter turn, go through sincospif.
//
// A warp owns a row's chunk of heads.  Lanes share a head as units of 2 x VE channels (the two sides of VE
// pairs), so norm, rotation and gradients stay in registers and each value is read and written once; the
// row's cosines are computed once per chunk by the whole warp and handed round through shared memory.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "cache.h"
#include "common.cuh"
#include "rope.h"

namespace bpa {
namespace {

constexpr int kWarps = 8, kMaxD = 512;

// VE channels, as they stand in memory
template <typename E, int VE>
struct Raw;
template <>
struct Raw<__nv_bfloat16, 8> {
    uint4 v;
    BPA_DEV void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
    BPA_DEV void zero() { v = make_uint4(0, 0, 0, 0); }
    BPA_DEV void get(float* f) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(w[i] << 16);
            f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
    static BPA_DEV void store(__nv_bfloat16* p, const float* f) {
        *reinterpret_cast<uint4*>(p) =
            make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
    }
};
template <>
struct Raw<float, 4> {
    float4 v;
    BPA_DEV void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
    BPA_DEV void zero() { v = make_float4(0.f, 0.f, 0.f, 0.f); }
    BPA_DEV void get(float* f) const {
        f[0] = v.x;
        f[1] = v.y;
        f[2] = v.z;
        f[3] = v.w;
    }
    static BPA_DEV void store(float* p, const float* f) { *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]); }
};
template <typename E>
struct Raw<E, 1> {
    E v;
    BPA_DEV void load(const E* p) { v = *p; }
    BPA_DEV void zero() { v = static_cast<E>(0.f); }
    BPA_DEV void get(float* f) const { f[0] = static_cast<float>(v); }
    static BPA_DEV void store(E* p, const float* f) { *p = static_cast<E>(f[0]); }
};

// inv_freq as a fraction of a turn, 64 bits behind the point.  1 / 2 pi in two doubles: the product with a
// float32 is exact but for 2^-100 or so, and 2^-64 of a turn times 2^31 is 2^-33.
BPA_DEV uint64_t turn_of(float f) {
    constexpr double hi = 0.15915494309189535, lo = -9.839338337591243e-18;   // 1 / 2 pi
    const double x = f, a = x * hi, b = fma(x, hi, -a) + x * lo;
    return static_cast<uint64_t>(__double2ll_rn((a - rint(a)) * 18446744073709551616.0)) +
           static_cast<uint64_t>(__double2ll_rn(b * 18446744073709551616.0));
}
BPA_DEV float2 cos_sin(uint64_t turn, int pos) {
    const uint32_t x = static_cast<uint32_t>((turn * static_cast<uint64_t>(pos)) >> 32);
    const uint32_t q = (x + (1u << 29)) >> 30;                   // the nearest quarter turn
    float s, c;
    sincospif(static_cast<float>(static_cast<int>(x - (q << 30))) * 4.656612873077393e-10f, &s, &c);
    const float u = q & 1 ? s : c, v = q & 1 ? c : s;
    return make_float2((q + 1) & 2 ? -u : u, q & 2 ? -v : v);
}

// Where a lane's unit u of a head lies: channels a.. and b.. (b may be past an odd d), its first pairs.
struct Unit {
    int a, b, pa, pb;                  // pairs of side a (and b, where a pair lies within a side); -1: not rotated
};
template <int VE, bool INTER>
BPA_DEV Unit unit_of(int u, int d, int rot) {
    if (INTER && VE > 1) {             // neighbours within a side
        const int a = VE * u, b = d / 2 + VE * u;
        return {a, b, a < rot ? a / 2 : -1, b < rot ? b / 2 : -1};
    }
    if (INTER) return {2 * u, 2 * u + 1, 2 * u < rot ? u : -1, -1};
    const int half = rot / (2 * VE);
    if (u < half) return {VE * u, rot / 2 + VE * u, VE * u, -1};
    const int a = rot + 2 * VE * (u - half);
    return {a, a + VE, -1, -1};
}

// The rotation of a unit, forward (SGN 1) or back (-1); c, s: cosines and sines of its pairs.
template <int VE, bool INTER>
BPA_DEV void rotate(float (&v)[2][VE], const Unit& u, const float (&c)[VE], const float (&s)[VE], float sgn) {
    if (INTER && VE > 1) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const bool on = (h ? u.pb : u.pa) >= 0;
#pragma unroll
            for (int i = 0; i < VE / 2; ++i) {
                const float cc = c[h * (VE / 2) + i], ss = sgn * s[h * (VE / 2) + i];
                const float x = v[h][2 * i], y = v[h][2 * i + 1];
                if (on) {
                    v[h][2 * i] = x * cc - y * ss;
                    v[h][2 * i + 1] = y * cc + x * ss;
                }
            }
        }
    } else {
        const bool on = u.pa >= 0;
#pragma unroll
        for (int i = 0; i < VE; ++i) {
            const float x = v[0][i], y = v[1][i], ss = sgn * s[i];
            if (on) {
                v[0][i] = x * c[i] - y * ss;
                v[1][i] = y * c[i] + x * ss;
            }
        }
    }
}

// Sums over the `lanes` lanes of a head, the same bits on each.
BPA_DEV float head_sum(float x, int lanes) {
    for (int o = lanes >> 1; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
// 1 / sqrt(mean x^2 + eps) of a head whose squares leave float32's range (or come close): the head is
// scaled by a power of two, which stays in v; the factor belongs to the scaled values.
template <int VE, int U>
BPA_DEV float far_norm(float (&v)[U][2][VE], float& scale, int lanes, int d, float eps) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < U * 2 * VE; ++i) top = fmaxf(top, fabsf((&v[0][0][0])[i]));
    for (int o = lanes >> 1; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const int e = top > 0.f && top < INFINITY ? min(max(127 - static_cast<int>(__float_as_uint(top) >> 23), -126), 60) : 0;
    scale = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < U * 2 * VE; ++i) {
        float& x = (&v[0][0][0])[i];
        x *= scale;
        ss = fmaf(x, x, ss);
    }
    return rsqrtf(head_sum(ss, lanes) / d + eps * scale * scale);
}
constexpr float kNear = 1.2676506e30f;  // 2^100: mean squares between its inverse and it need no scaling

// A side's heads in chunks, the rows in order: item = row * chunks + chunk.
struct Split {
    int lanes, per, chunk, chunks[2];  // lanes of a head, heads side by side, heads of a chunk, chunks of a row
};

template <typename E, int VE, int U, bool INTER, bool BWD, int HB>
__global__ void __launch_bounds__(32 * kWarps) k_rope(const RopeArgs a, const Split sp) {
    __shared__ uint64_t s_turn[kMaxD / 2];
    __shared__ float2 s_cs[kWarps][kMaxD / 2];
    extern __shared__ float s_dw[];    // BWD: [kWarps][d]
    using R = Raw<E, VE>;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lanes = sp.lanes, li = lane % lanes, gi = lane / lanes;
    const int pairs = a.rot / 2, units = (a.d + 2 * VE - 1) / (2 * VE);
    wait_for_previous();
    for (int i = threadIdx.x; i < pairs; i += 32 * kWarps) s_turn[i] = turn_of(a.freq[i]);
    __syncthreads();
    const int64_t rows = static_cast<int64_t>(a.B) * a.S, W = static_cast<int64_t>(gridDim.x) * kWarps;
    const int64_t me = static_cast<int64_t>(blockIdx.x) * kWarps + warp;
    Unit un[U];
#pragma unroll
    for (int u = 0; u < U; ++u) un[u] = unit_of<VE, INTER>(li + u * lanes, a.d, a.rot);

    int64_t from = 0;                  // items in front of this side's
    for (int side = 0; side < 2; ++side) {
        const RopeSide& t = a.side[side];
        const int64_t items = rows * sp.chunks[side];
        float w[U][2][VE], dw[U][2][VE];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    const int c = (h ? un[u].b : un[u].a) + i;
                    w[u][h][i] = t.w && li + u * lanes < units && c < a.d ? t.w[c] : 1.f;
                    dw[u][h][i] = 0.f;
                }
        // the warps take the items of both sides in turn
        for (int64_t it = (me - from % W + W) % W; it < items; it += W) {
            const int64_t row = it / sp.chunks[side];
            const int h0 = static_cast<int>(it - row * sp.chunks[side]) * sp.chunk, h1 = min(t.H, h0 + sp.chunk);
            const int b = static_cast<int>(row / a.S), s = static_cast<int>(row - static_cast<int64_t>(b) * a.S);
            const int pos = a.pos ? a.pos[row] : s;
            if (pos < 0 && !BWD) continue;
            __syncwarp();
            for (int i = lane; i < pairs; i += 32) s_cs[warp][i] = cos_sin(s_turn[i], max(pos, 0));
            __syncwarp();
            float c[U][VE], sn[U][VE];
#pragma unroll
            for (int u = 0; u < U; ++u)
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    int p = un[u].pa < 0 ? -1 : un[u].pa + i;
                    if (INTER && VE > 1) p = i < VE / 2 ? p : un[u].pb < 0 ? -1 : un[u].pb + i - VE / 2;
                    const float2 x = p >= 0 && p < pairs ? s_cs[warp][p] : make_float2(1.f, 0.f);
                    c[u][i] = x.x;
                    sn[u][i] = x.y;
                }
            const E* x0 = static_cast<const E*>(t.x) + b * t.xs[0] + s * t.xs[1];
            const E* g0 = static_cast<const E*>(t.dy) + b * t.ys[0] + s * t.ys[1];
            E* y0 = static_cast<E*>(t.y) + b * (BWD ? t.xs[0] : t.ys[0]) + s * (BWD ? t.xs[1] : t.ys[1]);
            const int64_t y_head = BWD ? t.xs[2] : t.ys[2];
            for (int hh = h0 + gi; __any_sync(0xffffffffu, hh < h1); hh += HB * sp.per) {
                R rx[HB][U][2], rg[HB][U][2];
#pragma unroll
                for (int j = 0; j < HB; ++j)
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int ch = h ? un[u].b : un[u].a, head = hh + j * sp.per;
                            const bool on = head < h1 && li + u * lanes < units && ch < a.d && pos >= 0;
                            rx[j][u][h].zero();
                            if (on) rx[j][u][h].load(x0 + head * t.xs[2] + ch);
                            if (BWD) {
                                rg[j][u][h].zero();
                                if (on) rg[j][u][h].load(g0 + head * t.ys[2] + ch);
                            }
                        }
#pragma unroll
                for (int j = 0; j < HB; ++j) {
                    const int head = hh + j * sp.per;
                    float v[U][2][VE], g[U][2][VE];
                    float ss = 0.f, xg = 0.f;
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            rx[j][u][h].get(v[u][h]);
                            if (BWD) rg[j][u][h].get(g[u][h]);
                        }
                    if (BWD) {
#pragma unroll
                        for (int u = 0; u < U; ++u) rotate<VE, INTER>(g[u], un[u], c[u], sn[u], -1.f);
                    }
                    if (a.norm) {
#pragma unroll
                        for (int i = 0; i < U * 2 * VE; ++i) {
                            const float x = (&v[0][0][0])[i];
                            ss = fmaf(x, x, ss);
                            if (BWD) xg = fmaf(x * (&w[0][0][0])[i], (&g[0][0][0])[i], xg);
                        }
                        const float mean = head_sum(ss, lanes) / a.d + a.eps;
                        float r = rsqrtf(mean), scale = 1.f;
                        if (!__all_sync(0xffffffffu, mean > 1.f / kNear && mean < kNear)) {
                            r = far_norm<VE, U>(v, scale, lanes, a.d, a.eps);
                            xg = 0.f;
#pragma unroll
                            for (int i = 0; i < U * 2 * VE; ++i)
                                if (BWD) xg = fmaf((&v[0][0][0])[i] * (&w[0][0][0])[i], (&g[0][0][0])[i], xg);
                        }
                        if (BWD) {
                            const float m = head_sum(xg, lanes) * r / a.d;
#pragma unroll
                            for (int i = 0; i < U * 2 * VE; ++i) {
                                const float xh = (&v[0][0][0])[i] * r, e = (&g[0][0][0])[i];
                                (&dw[0][0][0])[i] = fmaf(e, xh, (&dw[0][0][0])[i]);
                                (&v[0][0][0])[i] = (e * (&w[0][0][0])[i] - xh * m) * r * scale;
                            }
                        } else {
#pragma unroll
                            for (int i = 0; i < U * 2 * VE; ++i) (&v[0][0][0])[i] = (&v[0][0][0])[i] * r * (&w[0][0][0])[i];
                        }
                    } else if (BWD) {
#pragma unroll
                        for (int i = 0; i < U * 2 * VE; ++i) (&v[0][0][0])[i] = (&g[0][0][0])[i];
                    }
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        if (!BWD) rotate<VE, INTER>(v[u], un[u], c[u], sn[u], 1.f);
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int ch = h ? un[u].b : un[u].a;
                            if (head < h1 && li + u * lanes < units && ch < a.d) R::store(y0 + head * y_head + ch, v[u][h]);
                        }
                    }
                }
            }
        }
        from += items;
        if (!BWD) continue;
        // the warps' sums, then the block's, in a fixed order
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    float x = dw[u][h][i];
                    for (int o = 16; o >= lanes; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                    const int ch = (h ? un[u].b : un[u].a) + i;
                    if (gi == 0 && li + u * lanes < units && ch < a.d) s_dw[warp * a.d + ch] = x;
                }
        __syncthreads();
        for (int ch = threadIdx.x; ch < a.d; ch += 32 * kWarps) {
            float x = 0.f;
#pragma unroll
            for (int k = 0; k < kWarps; ++k) x += s_dw[k * a.d + ch];
            a.part[(static_cast<int64_t>(blockIdx.x) * 2 + side) * a.d + ch] = x;
        }
    }
}

// dw = the blocks' sums added up in a fixed order, in 64 bits: 32 channels a block, 8 threads to a channel.
__global__ void __launch_bounds__(256) k_rope_dw(const RopeArgs a, int blocks) {
    __shared__ double s_sum[8][32];
    wait_for_previous();
    if (blockIdx.x == 0 && threadIdx.x < 2) a.status[threadIdx.x] = 0;
    const int ch = blockIdx.x * 32 + (threadIdx.x & 31), k = threadIdx.x >> 5;
    double x = 0.0;
    if (ch < 2 * a.d)
        for (int b = k; b < blocks; b += 8) x += a.part[static_cast<int64_t>(b) * 2 * a.d + ch];
    s_sum[k][threadIdx.x & 31] = x;
    __syncthreads();
    if (k || ch >= 2 * a.d) return;
#pragma unroll
    for (int i = 1; i < 8; ++i) x += s_sum[i][threadIdx.x];
    const int side = ch >= a.d;
    if (a.side[side].dw) a.side[side].dw[ch - side * a.d] = static_cast<float>(x);
}

int sm_count() {
    static std::atomic<int> cached[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
    n = cached[dev].load(std::memory_order_relaxed);
    if (n > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 1;
    cached[dev].store(n, std::memory_order_relaxed);
    return n;
}

template <typename E, int VE, int U, bool BWD>
cudaError_t launch(const RopeArgs& a, cudaStream_t s) {
    constexpr int HB = 1;
    Split sp;
    const int units = (a.d + 2 * VE - 1) / (2 * VE);
    sp.lanes = 1;
    while (sp.lanes < 32 && sp.lanes < units) sp.lanes *= 2;
    sp.per = 32 / sp.lanes;
    const int64_t rows = static_cast<int64_t>(a.B) * a.S, most = static_cast<int64_t>(sm_count()) * 4 * kWarps;
    const int H = a.side[0].H + a.side[1].H;
    // heads of a chunk: enough chunks for every warp of the GPU, each of whole rounds of heads
    const int64_t rounds = rows * ((H + sp.per - 1) / sp.per) / most;
    sp.chunk = sp.per * static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(rounds, (H + sp.per - 1) / sp.per)));
    int64_t items = 0;
    for (int i = 0; i < 2; ++i) {
        sp.chunks[i] = (a.side[i].H + sp.chunk - 1) / sp.chunk;
        items += rows * sp.chunks[i];
    }
    const int blocks = static_cast<int>(std::min<int64_t>({(items + kWarps - 1) / kWarps, most / kWarps, kRopeMaxBlocks}));
    const size_t smem = BWD ? sizeof(float) * kWarps * a.d : 0;
    cudaError_t e = cudaSuccess;
    if (blocks > 0) {
        auto kernel = a.interleaved ? k_rope<E, VE, U, true, BWD, HB> : k_rope<E, VE, U, false, BWD, HB>;
        e = launch_early(dim3(blocks), dim3(32 * kWarps), smem, s, kernel, a, sp);
    }
    if (!BWD || e != cudaSuccess) return e;
    return launch_early(dim3((2 * a.d + 31) / 32), dim3(256), 0, s, k_rope_dw, a, blocks);
}

template <typename E, bool BWD>
cudaError_t by_shape(const RopeArgs& a, cudaStream_t s) {
    return a.d <= 128 ? launch<E, 1, 2, BWD>(a, s) : launch<E, 1, 8, BWD>(a, s);
}

}  // namespace

cudaError_t launch_rope_fwd(const RopeArgs& a, cudaStream_t s) {
    return a.dtype == BPA_BF16 ? by_shape<__nv_bfloat16, false>(a, s) : by_shape<float, false>(a, s);
}
cudaError_t launch_rope_bwd(const RopeArgs& a, cudaStream_t s) {
    return a.dtype == BPA_BF16 ? by_shape<__nv_bfloat16, true>(a, s) : by_shape<float, true>(a, s);
}

}  // namespace bpa
