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
// A warp owns a row's chunk of heads.  Lanes share a head as units of 16 bytes (the two sides of VE pairs), so norm,
// rotation and gradients stay in registers and each value is read and written once; the row's cosines are
// computed once per chunk by the whole warp and handed round through shared memory.  Arithmetic goes two
// float32 at a time, sums through float32, and what is read is on its way three rounds of heads ahead
// (cp.async into each lane's own places, which costs no registers).
//
// Bounded by HBM where there is much: forward of 8,192 rows x 136 heads x 128 bf16 channels 94 us, 6.1 TB/s (90 % of the
// measured copy); backward of 8,192 x 40 heads 49.4 us, 5.1 TB/s, of which 3 are the second launch, which adds up the
// blocks' sums of dw (bound by its instructions and the registers of the weights' sums, four blocks an SM; scalar
// arithmetic 56 us).  By latency where there is little: 64 rows x 40 heads 4.5 us, backward of 999 rows x 6 heads 8.6.
// Forward of 8,192 x 40 heads 35.2 us; float32 57.4, backward 88.3 (5.8 and 5.7 TB/s).
// Shapes that 16-byte units do not fit go element by element (k_rope_any): the two large ones above 315 and 211 us; 8,192 x 40
// heads of 80 channels with 20 or 40 rotated 145 us, backward 180 (floors 15.5 and 23.2), of 96 with 24 147 and 184.  Bound by
// latency: sixteen warps an SM, each of which waits for one head's loads (44 % of its time forward, 33 % backward) and then
// for its shuffles, use 43 and 50 % of the issue slots and a tenth of the L2's rate.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "cache.h"
#include "common.cuh"
#include "rope.h"

namespace bpa {
namespace {

constexpr int kWarps = 4, kMaxD = 512;

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

// Sums over the `lanes` lanes of a head, the same bits on each.
BPA_DEV float head_sum(float x, int lanes) {
#pragma unroll
    for (int o = 16; o; o >>= 1)
        if (o < lanes) x += __shfl_xor_sync(0xffffffffu, x, o);
    return x;
}
BPA_DEV float head_max(float x, int lanes) {
    for (int o = lanes >> 1; o; o >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}
// A mean square (with eps) between 1 / kNear and kNear needs no scaling (k_rope's backward pass sums weight x gradient x
// value before it has the root: 512 values of up to 2^25 leave room for weight x gradient up to 2^90); otherwise the
// head is scaled by a power of two first: the larger of its largest value and sqrt(eps) to [1, 2), so that neither the
// squares nor eps times the square of the scale leave float32's range (eps is at least 2^-126, so the scale at most 2^63).
constexpr float kNear = 1.0995116e12f;  // 2^40
BPA_DEV bool near(float mean) { return mean > 1.f / kNear && mean < kNear; }
BPA_DEV float far_scale(float top, int most) {
    const int e = top > 0.f && top < INFINITY ? min(max(127 - static_cast<int>(__float_as_uint(top) >> 23), -126), most) : 0;
    return __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
}

// A side's heads in chunks, the rows in order: item = row * chunks + chunk.
struct Split {
    int lanes, per, chunk, chunks[2];  // lanes of a head, heads side by side, heads of a chunk, chunks of a row
};

// What the warps share: the turns of all frequencies, each warp's cosines and sines, sums of dw.
struct Shared {
    uint64_t turn[kMaxD / 2];
    float2 cs[kWarps][kMaxD / 2];
};

// The items of one warp: every W-th of a side's, the next side's behind them.
struct Walk {
    int rows, W, me, chunks, down, along, row, at;
    BPA_DEV Walk(const RopeArgs& a) : rows(a.B * a.S), W(gridDim.x * kWarps), me(blockIdx.x * kWarps + (threadIdx.x >> 5)) {}
    BPA_DEV void begin(int n) {        // W items are `down` rows and `along` chunks
        chunks = n;
        down = n ? W / n : 0;
        along = n ? W % n : 0;
        row = n ? me / n : rows;
        at = n ? me % n : 0;
    }
    BPA_DEV bool there() const { return row < rows; }
    BPA_DEV void next() {
        const bool over = at + along >= chunks;
        row += down + over;
        at += along - (over ? chunks : 0);
    }
    BPA_DEV void end() {
        me -= static_cast<int>(static_cast<int64_t>(rows) * chunks % W);
        if (me < 0) me += W;
    }
};

// The block's sums of dw for one side from its warps', in a fixed order; s_dw [kWarps][d] is filled by `put`.
template <typename F>
BPA_DEV void block_dw(const RopeArgs& a, int side, float* s_dw, F put) {
    __syncthreads();
    put();
    __syncthreads();
    for (int ch = threadIdx.x; ch < a.d; ch += 32 * kWarps) {
        float x = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) x += s_dw[k * a.d + ch];
        a.part[(static_cast<int64_t>(blockIdx.x) * 2 + side) * a.d + ch] = x;
    }
}

// ---- any shape and alignment: a lane holds one or more pairs (channels a and b), element by element
template <typename E, int U, bool INTER, bool BWD>
__global__ void __launch_bounds__(32 * kWarps) k_rope_any(const RopeArgs a, const Split sp) {
    __shared__ Shared sh;
    extern __shared__ float s_dw[];    // BWD: [kWarps][d]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lanes = sp.lanes, li = lane % lanes, gi = lane / lanes, pairs = a.rot / 2;
    wait_for_previous();
    for (int i = threadIdx.x; i < pairs; i += 32 * kWarps) sh.turn[i] = turn_of(a.freq[i]);
    __syncthreads();
    int ch[U][2];                      // channels past d: none
    bool on[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int i = li + u * lanes;
        on[u] = i < pairs;
        ch[u][0] = INTER || !on[u] ? 2 * i : i;
        ch[u][1] = INTER || !on[u] ? 2 * i + 1 : i + pairs;
    }
    Walk walk(a);
    for (int side = 0; side < 2; ++side) {
        const RopeSide& t = a.side[side];
        float w[U][2], dw[U][2];
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                w[u][h] = t.w && ch[u][h] < a.d ? t.w[ch[u][h]] : 1.f;
                dw[u][h] = 0.f;
            }
        for (walk.begin(sp.chunks[side]); walk.there(); walk.next()) {
            const int row = walk.row, h0 = walk.at * sp.chunk, h1 = min(t.H, h0 + sp.chunk);
            const int b = row / a.S, s = row - b * a.S, pos = a.pos ? a.pos[row] : s;
            if (pos < 0 && !BWD) continue;
            __syncwarp();
            for (int i = lane; i < pairs; i += 32) sh.cs[warp][i] = cos_sin(sh.turn[i], max(pos, 0));
            __syncwarp();
            const E* x0 = static_cast<const E*>(t.x) + b * t.xs[0] + s * t.xs[1];
            const E* g0 = static_cast<const E*>(t.dy) + b * t.ys[0] + s * t.ys[1];
            E* y0 = static_cast<E*>(t.y) + b * (BWD ? t.xs[0] : t.ys[0]) + s * (BWD ? t.xs[1] : t.ys[1]);
            const int64_t y_head = BWD ? t.xs[2] : t.ys[2];
            for (int head = h0 + gi; __any_sync(0xffffffffu, head < h1); head += sp.per) {
                float v[U][2], g[U][2], ss = 0.f, top = 0.f;
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const float2 cs = on[u] ? sh.cs[warp][li + u * lanes] : make_float2(1.f, 0.f);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const bool there = head < h1 && ch[u][h] < a.d && pos >= 0;
                        v[u][h] = there && (a.norm || !BWD) ? static_cast<float>(x0[head * t.xs[2] + ch[u][h]]) : 0.f;
                        g[u][h] = BWD && there ? static_cast<float>(g0[head * t.ys[2] + ch[u][h]]) : 0.f;
                        ss = fmaf(v[u][h], v[u][h], ss);
                        top = fmaxf(top, fabsf(v[u][h]));
                    }
                    if (BWD && on[u]) {
                        const float p = g[u][0], q = g[u][1];
                        g[u][0] = p * cs.x + q * cs.y;
                        g[u][1] = q * cs.x - p * cs.y;
                    }
                }
                if (a.norm) {
                    const float mean = head_sum(ss, lanes) / a.d + a.eps;
                    float r = rsqrtf(mean), scale = 1.f;
                    if (!__all_sync(0xffffffffu, near(mean))) {
                        scale = far_scale(head_max(top, lanes), a.far);
                        ss = 0.f;
#pragma unroll
                        for (int u = 0; u < U; ++u)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                v[u][h] *= scale;
                                ss = fmaf(v[u][h], v[u][h], ss);
                            }
                        r = rsqrtf(head_sum(ss, lanes) / a.d + a.eps * scale * scale);
                    }
                    float xg = 0.f;
#pragma unroll
                    for (int u = 0; u < U; ++u)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            v[u][h] *= r;                          // xh
                            if (!BWD) v[u][h] *= w[u][h];
                            else {
                                dw[u][h] = fmaf(g[u][h], v[u][h], dw[u][h]);
                                g[u][h] *= w[u][h];
                                xg = fmaf(g[u][h], v[u][h], xg);
                            }
                        }
                    if (BWD) {
                        const float m = head_sum(xg, lanes) / a.d;
#pragma unroll
                        for (int u = 0; u < U; ++u)
#pragma unroll
                            for (int h = 0; h < 2; ++h) g[u][h] = (g[u][h] - v[u][h] * m) * r * scale;
                    }
                }
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (!BWD) {
                        const float p = v[u][0], q = v[u][1];
                        const float2 cs = on[u] ? sh.cs[warp][li + u * lanes] : make_float2(1.f, 0.f);
                        g[u][0] = on[u] ? p * cs.x - q * cs.y : p;
                        g[u][1] = on[u] ? q * cs.x + p * cs.y : q;
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h)
                        if (head < h1 && ch[u][h] < a.d) y0[head * y_head + ch[u][h]] = static_cast<E>(g[u][h]);
                }
            }
        }
        walk.end();
        if (BWD)
            block_dw(a, side, s_dw, [&] {
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float x = dw[u][h];
                        for (int o = 16; o >= lanes; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
                        if (gi == 0 && ch[u][h] < a.d) s_dw[warp * a.d + ch[u][h]] = x;
                    }
            });
    }
}

// ---- units of 16 bytes: a lane holds two (sides 0 and 1), the two sides of VE pairs or, interleaved, VE
// pairs in themselves; all arithmetic on pairs of float32
template <typename E>
struct Unit;
template <>
struct Unit<__nv_bfloat16> {
    static constexpr int VE = 8;
    uint4 v;
    BPA_DEV void get(uint64_t (&f)[4]) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    }
    BPA_DEV void set(const uint64_t (&f)[4]) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float x, y;
            f2_unpack(f[i], x, y);
            w[i] = pack_bf16(x, y);
        }
        v = make_uint4(w[0], w[1], w[2], w[3]);
    }
};
template <>
struct Unit<float> {
    static constexpr int VE = 4;
    uint4 v;
    BPA_DEV void get(uint64_t (&f)[2]) const {
        f[0] = f2_pack(__uint_as_float(v.x), __uint_as_float(v.y));
        f[1] = f2_pack(__uint_as_float(v.z), __uint_as_float(v.w));
    }
    BPA_DEV void set(const uint64_t (&f)[2]) {
        float x, y, z, w;
        f2_unpack(f[0], x, y);
        f2_unpack(f[1], z, w);
        v = make_uint4(__float_as_uint(x), __float_as_uint(y), __float_as_uint(z), __float_as_uint(w));
    }
};
BPA_DEV uint64_t swapped(uint64_t v) {
    float x, y;
    f2_unpack(v, x, y);
    return f2_pack(y, x);
}
BPA_DEV float sum2(uint64_t v) {
    float x, y;
    f2_unpack(v, x, y);
    return x + y;
}
BPA_DEV float max2(uint64_t v) {
    float x, y;
    f2_unpack(v, x, y);
    return fmaxf(fabsf(x), fabsf(y));
}

// This lane's place in a head: first channels of its sides, first pairs of them; -1: not rotated.
struct Place {
    int ch[2], pair[2];
};
template <int VE, bool INTER>
BPA_DEV Place place_of(int u, int d, int rot) {
    if (INTER) {
        const int a = VE * u, b = d / 2 + VE * u;
        return {{a, b}, {a < rot ? a / 2 : -1, b < rot ? b / 2 : -1}};
    }
    const int half = rot / (2 * VE), a = rot + 2 * VE * (u - half);
    return u < half ? Place{{VE * u, rot / 2 + VE * u}, {VE * u, VE * u}} : Place{{a, a + VE}, {-1, -1}};
}
// The rotation of element pair i of side h: y = v P + o Q with o the other side's elements and P = (c, c'), Q =
// (-s, -s') on side 0, (s, s') on side 1; interleaved, o is the neighbour, P = (c, c), Q = (-s, s).
// Loaded as (P, Q of side 1): what the sides share is kept once.
template <bool INTER>
BPA_DEV void turn_at(const float2* cs, const Place& pl, int h, int i, uint64_t& P, uint64_t& Q) {
    P = f2_pack(1.f, 1.f);
    Q = 0;
    if (pl.pair[h] < 0) return;
    if (INTER) {
        const float2 x = cs[pl.pair[h] + i];
        P = f2_pack(x.x, x.x);
        Q = f2_pack(-x.y, x.y);
    } else {
        const float4 x = *reinterpret_cast<const float4*>(cs + pl.pair[h] + 2 * i);
        P = f2_pack(x.x, x.z);
        Q = f2_pack(x.y, x.w);
    }
}
BPA_DEV uint64_t minus2(uint64_t v) { return v ^ 0x8000000080000000ull; }

// What a warp reads is on its way kStages - 1 rounds ahead (a round: `per` heads side by side), across rows and
// items, in shared memory and not in registers: each lane copies the 16-byte units that it will read itself, so
// nothing but its own copies has to be waited for.
constexpr int kStages = 4;
BPA_DEV void copy16(uint32_t to, const void* from, bool there) {   // zeros where nothing is there
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(there ? 16 : 0) : "memory");
}
BPA_DEV void copies_close() { asm volatile("cp.async.commit_group;" ::: "memory"); }
BPA_DEV void copies_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory"); }

// What the reading side leaves for the one that computes: the round's elements in the output, heads left of the item.
struct Round {
    int64_t out;
    int pos;
    int left;                          // 0: the end; kFirst: the item's first round
};
constexpr int kFirst = 1 << 30;

// LANES: lanes of a head, 0 for sp.lanes.  Known, the sums' steps and the places need no predicates: backward 51.7 -> 48.7
// us (8,192 rows x 40 heads of 128 channels); forward, which waits for memory alone, 100 -> 105.
template <typename E, bool INTER, bool BWD, int LANES>
__global__ void __launch_bounds__(32 * kWarps, 4) k_rope(const RopeArgs a, const Split sp, const float inv_d) {
    constexpr int VE = Unit<E>::VE, N = VE / 2, PIECES = BWD ? 4 : 2;
    __shared__ __align__(16) Shared sh;
    __shared__ __align__(16) uint4 s_ring[kWarps][kStages][PIECES][32];
    __shared__ __align__(16) Round s_round[kWarps][kStages];
    float* s_dw = reinterpret_cast<float*>(s_ring);               // [kWarps][d], when the rounds are over
    static_assert(sizeof s_ring >= sizeof(float) * kWarps * kMaxD, "sums of dw");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int lanes = LANES ? LANES : sp.lanes, li = lane % lanes, gi = lane / lanes, pairs = a.rot / 2;
    const bool mine = li < a.d / (2 * VE), part = a.rot < a.d;
    const Place pl = place_of<VE, INTER>(li, a.d, a.rot);
    const int other = pl.ch[1] - pl.ch[0];
    const uint32_t ring = smem_u32(&s_ring[warp][0][0][lane]);
    wait_for_previous();
    for (int i = threadIdx.x; i < pairs; i += 32 * kWarps) sh.turn[i] = turn_of(a.freq[i]);
    __syncthreads();
    Walk walk(a);
    for (int side = 0; side < 2; ++side) {
        const RopeSide& t = a.side[side];
        walk.begin(sp.chunks[side]);
        const int64_t x_round = t.xs[2] * sp.per, y_round = t.ys[2] * sp.per;
        const E* const x_lane = static_cast<const E*>(t.x) + gi * t.xs[2] + pl.ch[0];
        const E* const g_lane = static_cast<const E*>(t.dy) + gi * t.ys[2] + pl.ch[0];
        E* const to_lane = static_cast<E*>(t.y) + gi * (BWD ? t.xs[2] : t.ys[2]) + pl.ch[0];
        const E *x = nullptr, *g = nullptr;    // the round that is read next: this lane's units,
        int64_t out_at = 0;                    // the round's elements in the output,
        int left = 0, pos_at = 0;              // heads left of the item and its position
        auto open = [&]() {            // the item's first round
            const int h0 = walk.at * sp.chunk, b = walk.row / a.S, s = walk.row - b * a.S;
            left = min(t.H - h0, sp.chunk);
            pos_at = a.pos ? *(a.pos + walk.row) : s;
            const int64_t x_at = b * t.xs[0] + s * t.xs[1] + h0 * t.xs[2], y_at = b * t.ys[0] + s * t.ys[1] + h0 * t.ys[2];
            x = x_lane + x_at;
            if (BWD) g = g_lane + y_at;
            out_at = BWD ? x_at : y_at;
        };
        bool first = true;
        auto issue = [&](int st) {     // the next round into stage st
            if (left > 0) {
                const bool on = mine && gi < left && pos_at >= 0, on_x = on && (!BWD || a.norm);
                const uint32_t to = ring + st * (PIECES * 512);
                copy16(to, x, on_x);
                copy16(to + 512, x + other, on_x);
                if (BWD) {
                    copy16(to + 1024, g, on);
                    copy16(to + 1536, g + other, on);
                }
            }
            copies_close();
            if (lane == 0) s_round[warp][st] = {out_at, pos_at, left <= 0 ? 0 : first ? left | kFirst : left};
            if (left <= 0) return;
            left -= sp.per;
            x += x_round;
            if (BWD) g += y_round;
            out_at += BWD ? x_round : y_round;
            first = left <= 0;
            if (!first) return;
            walk.next();
            if (walk.there()) open();
        };
        if (walk.there()) open();
        for (int st = 0; st < kStages - 1; ++st) issue(st);
        uint64_t w[2][N], dw[2][N];
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const float* at = t.w + pl.ch[h] + 2 * i;
                w[h][i] = t.w && mine ? f2_pack(at[0], at[1]) : f2_pack(1.f, 1.f);
                dw[h][i] = 0;
            }
        // channels that are not rotated keep what they had (0 times an infinity beside them would not)
        auto rotated = [&](const uint64_t (&from)[2][N], uint64_t (&to)[2][N]) {
            if (!part) return;
#pragma unroll
            for (int h = 0; h < 2; ++h)
                if (pl.pair[h] < 0)
#pragma unroll
                    for (int i = 0; i < N; ++i) to[h][i] = from[h][i];
        };
        // the rotation's coefficients; forward: with the weights in them, so of either side
        constexpr int SIDES = INTER || !BWD ? 2 : 1;
        uint64_t P[SIDES][N], Q[SIDES][N];
        for (int st = 0;; st = st + 1 == kStages ? 0 : st + 1) {
            copies_wait();
            __syncwarp();              // the round's record is written
            const Round now = s_round[warp][st];
            if (now.left == 0) break;
            const int pos = now.pos;
            if (now.left & kFirst) {
                for (int i = lane; i < pairs; i += 32) sh.cs[warp][i] = cos_sin(sh.turn[i], max(pos, 0));
                __syncwarp();
#pragma unroll
                for (int h = 0; h < SIDES; ++h)
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        turn_at<INTER>(sh.cs[warp], pl, h, i, P[h][i], Q[h][i]);
                        if (!BWD) {
                            if (!INTER && h == 0) Q[h][i] = minus2(Q[h][i]);
                            P[h][i] = fmul2(P[h][i], w[h][i]);
                            Q[h][i] = fmul2(Q[h][i], INTER ? swapped(w[h][i]) : w[1 - h][i]);
                        }
                    }
            }
            uint64_t v[2][N], g[2][N];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                Unit<E> u;
                u.v = s_ring[warp][st][h][lane];
                u.get(v[h]);
                if (BWD) {
                    u.v = s_ring[warp][st][PIECES - 2 + h][lane];
                    u.get(g[h]);
                }
            }
            if (BWD) {                 // turned back
                uint64_t y[2][N];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const uint64_t o = INTER ? swapped(g[h][i]) : g[1 - h][i], q = Q[h % SIDES][i];
                        y[h][i] = ffma2(g[h][i], P[h % SIDES][i], fmul2(INTER || h ? minus2(o) : o, q));
                    }
                rotated(g, y);
#pragma unroll
                for (int i = 0; i < 2 * N; ++i) g[i / N][i % N] = y[i / N][i % N];
            }
            float r = 1.f, scale = 1.f, m = 0.f;
            if (a.norm) {
                uint64_t ss = 0, xg = 0;
#pragma unroll
                for (int i = 0; i < 2 * N; ++i) {
                    ss = ffma2(v[i / N][i % N], v[i / N][i % N], ss);
                    if (BWD) xg = ffma2(fmul2(g[i / N][i % N], w[i / N][i % N]), v[i / N][i % N], xg);
                }
                const float mean = fmaf(head_sum(sum2(ss), lanes), inv_d, a.eps);
                r = rsqrtf(mean);
                if (!__all_sync(0xffffffffu, near(mean))) {
                    float top = 0.f;
#pragma unroll
                    for (int i = 0; i < 2 * N; ++i) top = fmaxf(top, max2(v[i / N][i % N]));
                    scale = far_scale(head_max(top, lanes), a.far);
                    ss = xg = 0;
#pragma unroll
                    for (int i = 0; i < 2 * N; ++i) {
                        v[i / N][i % N] = fmul2(v[i / N][i % N], f2_pack(scale, scale));
                        ss = ffma2(v[i / N][i % N], v[i / N][i % N], ss);
                        if (BWD) xg = ffma2(fmul2(g[i / N][i % N], w[i / N][i % N]), v[i / N][i % N], xg);
                    }
                    r = rsqrtf(fmaf(head_sum(sum2(ss), lanes), inv_d, a.eps * scale * scale));
                }
                if (BWD) m = -head_sum(sum2(xg), lanes) * r * inv_d;
            }
            const uint64_t r2 = f2_pack(r, r);
            if (!BWD) {
                // the norm first: values times weights may leave float32's range where the result does not
#pragma unroll
                for (int i = 0; i < 2 * N; ++i) v[i / N][i % N] = fmul2(v[i / N][i % N], r2);
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        g[h][i] = ffma2(v[h][i], P[h][i], fmul2(INTER ? swapped(v[h][i]) : v[1 - h][i], Q[h][i]));
                if (part) {
                    uint64_t vw[2][N];
#pragma unroll
                    for (int i = 0; i < 2 * N; ++i) vw[i / N][i % N] = fmul2(v[i / N][i % N], w[i / N][i % N]);
                    rotated(vw, g);
                }
            } else if (a.norm) {
                const uint64_t m2 = f2_pack(m, m), f2 = f2_pack(r * scale, r * scale);
#pragma unroll
                for (int i = 0; i < 2 * N; ++i) {
                    const uint64_t xh = fmul2(v[i / N][i % N], r2);
                    dw[i / N][i % N] = ffma2(g[i / N][i % N], xh, dw[i / N][i % N]);
                    g[i / N][i % N] = fmul2(ffma2(xh, m2, fmul2(g[i / N][i % N], w[i / N][i % N])), f2);
                }
            }
            if (mine && gi < (now.left & ~kFirst) && (BWD || pos >= 0)) {
                E* p = to_lane + now.out;
                Unit<E> z;
                z.set(g[0]);
                *reinterpret_cast<uint4*>(p) = z.v;
                z.set(g[1]);
                *reinterpret_cast<uint4*>(p + other) = z.v;
            }
            issue(st == 0 ? kStages - 1 : st - 1);                // the stage of the round before this one
        }
        walk.end();
        if (BWD)
            block_dw(a, side, s_dw, [&] {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        float z[2];
                        f2_unpack(dw[h][i], z[0], z[1]);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            for (int o = 16; o >= lanes; o >>= 1) z[e] += __shfl_xor_sync(0xffffffffu, z[e], o);
                            if (gi == 0 && mine) s_dw[warp * a.d + pl.ch[h] + 2 * i + e] = z[e];
                        }
                    }
            });
        __syncthreads();               // the ring may be written again
    }
}

// dw = the blocks' sums added up in a fixed order: 32 channels a block, 32 threads to a channel.
__global__ void __launch_bounds__(1024) k_rope_dw(const RopeArgs a, int blocks) {
    __shared__ float s_sum[32][33];
    wait_for_previous();
    if (blockIdx.x == 0 && threadIdx.x < 2) a.status[threadIdx.x] = 0;
    const int c = threadIdx.x & 31, ch = blockIdx.x * 32 + c, k = threadIdx.x >> 5;
    float x = 0.f;
    if (ch < 2 * a.d)
#pragma unroll 8
        for (int b = k; b < blocks; b += 32) x += a.part[static_cast<int64_t>(b) * 2 * a.d + ch];
    s_sum[k][c] = x;
    __syncthreads();
    x = s_sum[c][k];                   // a warp to a channel
#pragma unroll
    for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    const int out = blockIdx.x * 32 + k, side = out >= a.d;
    if (c == 0 && out < 2 * a.d && a.side[side].dw) a.side[side].dw[out - side * a.d] = x;
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

// units: of a head, each a lane's (or more than one for 32 lanes)
Split split_of(const RopeArgs& a, int units, int warps) {
    Split sp;
    sp.lanes = 4;
    while (sp.lanes < 32 && sp.lanes < units) sp.lanes *= 2;
    sp.per = 32 / sp.lanes;
    // Heads of a chunk: as many as leave an item for each of the GPU's warps, in whole rounds, but at most sixteen, so that the
    // warps read side by side: 8,192 rows of 128 + 8 heads 100 us without the limit, 93.7 with it, 93.9 with eight and 107
    // with four (each chunk works out its row's rotation again).
    const int64_t rounds = (a.side[0].H + sp.per - 1) / sp.per + (a.side[1].H + sp.per - 1) / sp.per;
    const int64_t each = static_cast<int64_t>(a.B) * a.S * rounds / warps;
    sp.chunk = sp.per * static_cast<int>(std::max<int64_t>(1, std::min<int64_t>(16, each)));
    for (int i = 0; i < 2; ++i) sp.chunks[i] = (a.side[i].H + sp.chunk - 1) / sp.chunk;
    return sp;
}

// Whether everything is aligned to units of 16 bytes, VE elements, and the rotated part made of them.
bool wide(const RopeArgs& a, int VE) {
    if (a.d > 64 * VE || a.d % (2 * VE) || (a.interleaved ? a.rot % VE : a.rot % (2 * VE))) return false;
    for (const RopeSide& t : a.side) {
        if (t.H == 0) continue;
        if ((reinterpret_cast<uintptr_t>(t.x) | reinterpret_cast<uintptr_t>(t.y) | reinterpret_cast<uintptr_t>(t.dy)) & 15) return false;
        for (int i = 0; i < 3; ++i)
            if (t.xs[i] % VE || t.ys[i] % VE) return false;
    }
    return true;
}

template <typename E, bool BWD>
cudaError_t launch(const RopeArgs& a, cudaStream_t s) {
    constexpr int VE = Unit<E>::VE;
    const bool vec = wide(a, VE);
    const int blocks_most = std::min(4 * sm_count(), kRopeMaxBlocks);
    const Split sp = split_of(a, vec ? a.d / (2 * VE) : (a.d + 1) / 2, blocks_most * kWarps);
    const int64_t items = static_cast<int64_t>(a.B) * a.S * (sp.chunks[0] + sp.chunks[1]);
    const int blocks = static_cast<int>(std::min<int64_t>((items + kWarps - 1) / kWarps, blocks_most));
    const size_t smem = BWD ? sizeof(float) * kWarps * a.d : 0;
    const float inv_d = 1.f / static_cast<float>(a.d);
    const dim3 grid(blocks), block(32 * kWarps);
    cudaError_t e = cudaSuccess;
    if (blocks == 0) {                 // no rows
    } else if (vec) {
        auto go = [&](auto kernel) { e = launch_early(grid, block, 0, s, kernel, a, sp, inv_d); };
        if constexpr (!BWD) {
            a.interleaved ? go(k_rope<E, true, false, 0>) : go(k_rope<E, false, false, 0>);
        } else {
            switch (sp.lanes) {
                case 4: a.interleaved ? go(k_rope<E, true, true, 4>) : go(k_rope<E, false, true, 4>); break;
                case 8: a.interleaved ? go(k_rope<E, true, true, 8>) : go(k_rope<E, false, true, 8>); break;
                case 16: a.interleaved ? go(k_rope<E, true, true, 16>) : go(k_rope<E, false, true, 16>); break;
                default: a.interleaved ? go(k_rope<E, true, true, 32>) : go(k_rope<E, false, true, 32>);
            }
        }
    } else if (a.d <= 128) {
        e = launch_early(grid, block, smem, s, a.interleaved ? k_rope_any<E, 2, true, BWD> : k_rope_any<E, 2, false, BWD>, a, sp);
    } else {
        e = launch_early(grid, block, smem, s, a.interleaved ? k_rope_any<E, 8, true, BWD> : k_rope_any<E, 8, false, BWD>, a, sp);
    }
    if (!BWD || e != cudaSuccess) return e;
    return launch_early(dim3((2 * a.d + 31) / 32), dim3(1024), 0, s, k_rope_dw, a, blocks);
}

}  // namespace

cudaError_t launch_rope_fwd(const RopeArgs& a, cudaStream_t s) {
    return a.dtype == BPA_BF16 ? launch<__nv_bfloat16, false>(a, s) : launch<float, false>(a, s);
}
cudaError_t launch_rope_bwd(const RopeArgs& a, cudaStream_t s) {
    return a.dtype == BPA_BF16 ? launch<__nv_bfloat16, true>(a, s) : launch<float, true>(a, s);
}

}  // namespace bpa
