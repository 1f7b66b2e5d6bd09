// cache_attn_mma.cu - attention of few query rows over the paged 8-bit cache (generation, drafts).
//
// An item is 16 RT query rows (row = token-in-request * G + q head in the group, so every row
// reads the same keys) of one request and kv head; its keys are walked in tiles of 64.  Codes are
// exact in fp16, so both products run on fp16 matrix instructions with float32 sums:
//   S = Q K^T   with each row of Q scaled by a power of two into fp16's range (bf16 rows lose
//               nothing above 2^-22 of the row's largest value; float32 rows go in as two halves);
//   z = S * (k scale of the page) * (row's scale), in log2 units; m and l from exp2(z - m), float32;
//   O += W V    with W = exp2(z + log2(v scale) - M + 9) in fp16, M the running maximum of
//               z + log2(v scale): the weight that a page's codes really have, so pages whose scales
//               lie far apart keep their precision.  M moves only when it grows by more than 6 (W <=
//               2^15); a weight below 2^-33 of the largest is dropped.  float32: W as two halves.
//
// Bounded by the bytes of K and V.  So the CTAs are persistent (two per SM) and each takes an equal
// share of all tiles of all items, whatever the lengths; a share may begin and end inside an item.
// Pieces of items go to the workspace as (m, l, O) and a second, small launch joins them in
// ascending order (its launch overlaps the first kernel: programmatic dependent launch), so nothing
// is added in an order that changes.  Per CTA one warp copies tiles by TMA (a page's rows at a
// time, swizzled) into a ring of stages and passes the page's scales beside them; four warps
// take 16 keys of a tile each (RT = 1), or each row tile's share of them.
//
// Layouts without bank conflicts or shuffles: channels are permuted between Q and K so that a lane's
// 16 consecutive bytes of a key feed four products, and keys (n odd: n ^ 4 within eight) so that
// the score fragment is the weight fragment and V's rows are read 16 bytes at a time; pairs of V's
// rows are interleaved by byte permutes on the way to fp16.
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "cache.h"
#include "common.cuh"

namespace bpa {
namespace {

constexpr int kTile = 64;             // keys per stage
constexpr int kNW = 4;                // consumer warps
constexpr int kThreads = 32 * (kNW + 1);
constexpr int kBatch = 8;             // tiles whose page ids and scales are fetched together
constexpr float kOff = 9.f;           // log2 of the largest fp16 weight right after M moved
constexpr float kLazy = 6.f;          // M moves when it grows by more

struct Rec {                          // what a CTA leaves for the join
    int lead, lead_ends;              // slot 0 holds a piece of an item begun by an earlier CTA; its last
    int trail;                        // slot 1 holds the first piece of an item that goes on
    int row0, hk, i0, nrows;          // that item
    uint32_t flags, where;            // this CTA's status
    int pad[3];
};
static_assert(sizeof(Rec) == 48, "record");

struct Work {
    CacheAttnArgs a;
    int RT, ctas;
    int vec_o;                        // o takes 16-byte stores
    Rec* recs;                        // [ctas]
    float2* ml;                       // [2 ctas][16 RT] (m in log2 units, l)
    float* part;                      // [2 ctas][16 RT][DVP] relative to m
};

struct Meta {
    int key0, len, n, row0, hk, i0, flags, pad;
    float ks[4], vs[4];               // scales of the tile's four 16-key chunks
};
enum { F_FIRST = 1, F_LAST = 2, F_LEAD = 4, F_TRAIL = 8 };

template <int DP, int DVP, bool SPLIT>
struct Cfg {
    static constexpr int RBK = DP < 128 ? DP : 128, RBV = DVP < 128 ? DVP : 128;   // bytes of a swizzled row
    static constexpr int HK = DP / RBK, HV = DVP / RBV;                            // 128-byte halves
    static constexpr int K_BYTES = kTile * DP, V_BYTES = kTile * DVP, STAGE = K_BYTES + V_BYTES;
    static constexpr bool Q_REGS = !SPLIT && DP <= 128;
    static constexpr int QF = DP / 16 * 512 * (SPLIT ? 2 : 1);                     // fragments of a row tile
    static constexpr int MERGE = 2 * (16 * DVP + 16 * 4) * 4;                      // two warps' states
    static constexpr int NS = DP + DVP <= 128 ? 8 : DP + DVP <= 192 ? 6 : DP + DVP <= 256 ? (SPLIT ? 4 : 5) : 4;
    static constexpr int OCC = DP <= 128 ? 2 : 1;
    static int smem(int RT) { return 1024 + NS * STAGE + MERGE + NS * (int)sizeof(Meta) + 256 + (Q_REGS ? 0 : RT * QF); }
};

BPA_DEV uint32_t cvt2(uint32_t two) {      // two e4m3 codes -> fp16 pair, exact
    uint32_t h;
    asm("{.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;}" : "=r"(h) : "r"(two));
    return h;
}
BPA_DEV uint32_t cvt2_hi(uint32_t four) {
    uint32_t h;
    asm("{.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, u;}" : "=r"(h) : "r"(four));
    return h;
}
BPA_DEV void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
BPA_DEV uint32_t h2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
BPA_DEV float2 h2f(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }
BPA_DEV uint4 lds128(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}
BPA_DEV uint2 lds64(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
    return v;
}
// byte offset of byte `col` of row `row` in a TMA-swizzled tile with rows of RB (64 or 128) bytes
template <int RB>
BPA_DEV uint32_t swz(int row, int col) {
    const uint32_t off = row * RB + col;
    return RB == 128 ? off ^ ((row & 7u) << 4) : off ^ (((row >> 1) & 3u) << 4);
}

BPA_DEV float ld_q(const float* p) { return __ldg(p); }
BPA_DEV float ld_q(const __nv_bfloat16* p) { return __bfloat162float(*p); }

// Key tiles of row group rg: first tile and count (at least one, so that rows without keys are
// written too; such a tile holds no allowed key).
struct Tiles {
    int first, n;
};
BPA_DEV Tiles tiles_of(const CacheAttnArgs& a, const Req& q, int rg, int rows_per) {
    const int i0 = rg * rows_per, i1 = min(q.n * a.G, i0 + rows_per) - 1;
    int lo, hi, x;
    row_keys(a, q, i0 / a.G, lo, x);
    row_keys(a, q, i1 / a.G, x, hi);
    if (lo > hi) return {0, 1};
    return {lo / kTile, hi / kTile - lo / kTile + 1};
}
BPA_DEV long long tiles_of_request(const CacheAttnArgs& a, const Req& q, int rows_per) {
    if (q.n == 0) return 0;
    long long n = 0;
    const int groups = (q.n * a.G + rows_per - 1) / rows_per;
    for (int rg = 0; rg < groups; ++rg) n += tiles_of(a, q, rg, rows_per).n;
    return n * a.Hkv;
}

template <int DP, int DVP, bool SPLIT>
__global__ void __launch_bounds__(kThreads, (Cfg<DP, DVP, SPLIT>::OCC))
    k_cache_attn_mma(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Work w) {
    using C = Cfg<DP, DVP, SPLIT>;
    using E = typename std::conditional<SPLIT, float, __nv_bfloat16>::type;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sb = smem_u32(smem);
    float* merge = reinterpret_cast<float*>(smem + C::NS * C::STAGE);
    Meta* meta = reinterpret_cast<Meta*>(smem + C::NS * C::STAGE + C::MERGE);
    const uint32_t bars = smem_u32(meta + C::NS);
    const uint32_t q_at = bars + 256;
    auto FULL = [&](int s) { return bars + 8u * s; };
    auto EMPTY = [&](int s) { return bars + 8u * (C::NS + s); };
    const uint32_t join_bar = bars + 16u * C::NS;
    static_assert(16 * C::NS + 8 <= 256, "barriers");
    __shared__ long long s_scan[kNW + 1];
    __shared__ int s_r;
    __shared__ long long s_off;
    __shared__ int s_abort;

    const CacheAttnArgs& a = w.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;
    const int rows_per = 16 * w.RT;
    Rec* rec = w.recs + cta;
    uint32_t* status = &rec->flags;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::NS; ++s) {
            mbar_init(FULL(s), 1);
            mbar_init(EMPTY(s), kNW);
        }
        mbar_init(join_bar, kNW);
        fence_mbar_init();
        s_abort = 0;
        s_r = -1;
        rec->flags = rec->where = 0;
        __threadfence();
    }
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    // ---- this CTA's share of the tiles: [begin, end) of the running sum over the requests
    const int per = (a.R + kThreads - 1) / kThreads, r0 = min(a.R, static_cast<int>(threadIdx.x) * per),
              r1 = min(a.R, r0 + per);
    long long mine = 0;
    for (int r = r0; r < r1; ++r) mine += tiles_of_request(a, request_of(a, r), rows_per);
    long long x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) s_scan[warp] = x;
    __syncthreads();
    long long total = 0, before = 0;
    for (int i = 0; i <= kNW; ++i) {
        if (i < warp) before += s_scan[i];
        total += s_scan[i];
    }
    before += x - mine;
    // with fewer tiles than CTAs the first ones take one each, so the pieces of an item lie side by side
    const int parts = static_cast<int>(min(total, static_cast<long long>(w.ctas)));
    const long long begin = cta < parts ? total * cta / parts : total, end = cta < parts ? total * (cta + 1) / parts : total;
    if (begin < end && begin >= before && begin < before + mine) {
        long long at = before;
        for (int r = r0; r < r1; ++r) {
            const long long n = tiles_of_request(a, request_of(a, r), rows_per);
            if (begin < at + n) {
                s_r = r;
                s_off = begin - at;
                break;
            }
            at += n;
        }
    }
    __syncthreads();

    if (warp == kNW) {
        // ---- producer: tiles of the share, item by item
        int r = s_r, stage = 0;
        uint32_t phase = 1;            // the ring starts empty
        long long left = end - begin;
        Rec out = {};
        bool ok = true;
        if (r >= 0) {
            const int BR = min(a.P, kTile);
            const uint32_t copy = static_cast<uint32_t>(BR) * (DP + DVP);
            Req rq = request_of(a, r);
            if (rq.bad && lane == 0) report(status, ST_CHECK, 0xCD1);
            int groups = (rq.n * a.G + rows_per - 1) / rows_per;
            long long off = s_off;
            const long long per_head = tiles_of_request(a, rq, rows_per) / a.Hkv;
            int hk = static_cast<int>(off / per_head), rg = 0;
            off -= hk * per_head;
            Tiles tl = tiles_of(a, rq, 0, rows_per);
            while (off >= tl.n) {
                off -= tl.n;
                tl = tiles_of(a, rq, ++rg, rows_per);
            }
            int t = static_cast<int>(off);
            while (left > 0 && ok) {
                const int te = static_cast<int>(min(static_cast<long long>(tl.n), t + left));
                const bool lead = t > 0, trail = te < tl.n;
                const int i0 = rg * rows_per;
                const int kind = lead ? F_LEAD : trail ? F_TRAIL : 0;
                if (lead) {
                    out.lead = 1;
                    out.lead_ends = !trail;
                } else if (trail) {
                    out.trail = 1;
                    out.row0 = rq.row0;
                    out.hk = hk;
                    out.i0 = i0;
                    out.nrows = min(rq.n * a.G - i0, rows_per);
                }
                const int32_t* table = a.table + static_cast<int64_t>(r) * a.max_pages;
                for (int b = t; b < te && ok; b += kBatch) {
                    // lane = tile of the batch * 4 + chunk of 16 keys
                    const int tile = b + (lane >> 2), chunk = lane & 3;
                    const int key = (tl.first + tile) * kTile + 16 * chunk;
                    int id = -1;
                    if (tile < te && key < rq.len) {
                        id = __ldg(table + key / a.P);
                        if (id < 0 || id >= a.num_pages) {
                            report(status, ST_CHECK, 0xCD0);
                            id = -1;
                        }
                    }
                    float ks = 0.f, vs = 0.f;
                    if (id >= 0) {
                        ks = __ldg(a.kscale + static_cast<int64_t>(id) * a.Hkv + hk);
                        vs = __ldg(a.vscale + static_cast<int64_t>(id) * a.Hkv + hk);
                    }
                    const int cnt = min(kBatch, te - b);
                    for (int j = 0; j < cnt; ++j) {
                        ok = mbar_wait(EMPTY(stage), phase, const_cast<volatile int*>(&s_abort), status, 0xCD2);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        const bool turn = (lane >> 2) == j;
                        const bool copies = turn && id >= 0 && (16 * chunk) % BR == 0;
                        const uint32_t n = __popc(__ballot_sync(0xffffffffu, copies));
                        Meta* m = meta + stage;
                        if (lane == 0) {
                            m->key0 = (tl.first + b + j) * kTile;
                            m->len = rq.len;
                            m->n = rq.n;
                            m->row0 = rq.row0;
                            m->hk = hk;
                            m->i0 = i0;
                            m->flags = kind | (b + j == t ? F_FIRST : 0) | (b + j == te - 1 ? F_LAST : 0);
                        }
                        if (turn) {
                            m->ks[chunk] = ks;
                            m->vs[chunk] = vs;
                        }
                        __syncwarp();
                        if (lane == 0) mbar_expect_tx(FULL(stage), n * copy);
                        __syncwarp();
                        if (copies) {
                            const uint32_t at = sb + stage * C::STAGE;
                            const int tok = key % a.P;
                            for (int h = 0; h < C::HK; ++h)
                                tma_load_4d(at + h * kTile * C::RBK + 16 * chunk * C::RBK, &tmK, FULL(stage), 128 * h, tok, hk, id);
                            for (int h = 0; h < C::HV; ++h)
                                tma_load_4d(at + C::K_BYTES + h * kTile * C::RBV + 16 * chunk * C::RBV, &tmV, FULL(stage),
                                            128 * h, tok, hk, id);
                        }
                        if (++stage == C::NS) {
                            stage = 0;
                            phase ^= 1;
                        }
                    }
                }
                left -= te - t;
                t = 0;
                if (left > 0) {        // the next item: row group, head, request
                    if (++rg == groups) {
                        rg = 0;
                        if (++hk == a.Hkv) {
                            hk = 0;
                            do {
                                if (++r >= a.R) break;      // only if the lengths changed during the call
                                rq = request_of(a, r);
                                if (rq.bad && rq.n && lane == 0) report(status, ST_CHECK, 0xCD1);
                            } while (rq.n == 0);
                            if (r >= a.R) {
                                if (lane == 0) report(status, ST_CHECK, 0xCD5);
                                break;
                            }
                            groups = (rq.n * a.G + rows_per - 1) / rows_per;
                        }
                    }
                    tl = tiles_of(a, rq, rg, rows_per);
                }
            }
        }
        // the copies in flight end before the CTA does: the consumers wait for them, and after a timeout
        // this warp (stages before `stage` hold this pass over the ring, the others the last one)
        if (!ok) {
            int never = 0;
            for (int s = 0; s < C::NS; ++s) mbar_wait(FULL(s), s < stage ? phase ^ 1 : phase, &never, status, 0xCD3);
        }
        if (lane == 0) {
            rec->lead = out.lead;
            rec->lead_ends = out.lead_ends;
            rec->trail = out.trail;
            rec->row0 = out.row0;
            rec->hk = out.hk;
            rec->i0 = out.i0;
            rec->nrows = out.nrows;
        }
        return;
    }

    // ---- consumers
    const int rt = warp % w.RT, slices = kNW / w.RT, slice = warp / w.RT;
    const int g = lane >> 2, j = lane & 3;
    const uint32_t my_q = q_at + rt * C::QF + lane * 16;
    uint32_t qf[C::Q_REGS ? DP / 16 : 1][4];
    float acc[DVP / 8][4];
    float m0, m1, M0, M1, l0, l1, f0 = 0.f, f1 = 0.f;
    int lo0 = 0, lo1 = 0, hi0 = 0, hi1 = 0, in_lo = 0, in_hi = 0, any_lo = 0, any_hi = 0;
    int stage = 0;
    uint32_t phase = 0, join_phase = 0;
    // a barrier of the consumers whose wait is bounded
    auto consumers_meet = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(join_bar);
        const bool met = mbar_wait(join_bar, join_phase, const_cast<volatile int*>(&s_abort), status, 0xCD6);
        join_phase ^= 1;
        return __all_sync(0xffffffffu, met) != 0;
    };
    for (long long t = begin; t < end; ++t) {
        if (!__all_sync(0xffffffffu, mbar_wait(FULL(stage), phase, const_cast<volatile int*>(&s_abort), status, 0xCD4))) return;
        const Meta* mt = meta + stage;
        const int flags = mt->flags, key0 = mt->key0, len = mt->len;
        if (flags & F_FIRST) {
            // ---- a new item: this warp's 16 rows of q as fp16 fragments, scaled by a power of two
            const Req rq = {mt->row0, mt->n, len, false};
            const int hk = mt->hk, nr = rq.n * a.G;
            float fac[2];
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                const int ri = mt->i0 + rt * 16 + g + 8 * half;
                const bool there = ri < nr;
                const int tok = there ? ri / a.G : 0;
                int lo = 0, hi = INT_MAX;          // a row that is not there masks nothing (q = 0: z = 0)
                if (there) row_keys(a, rq, tok, lo, hi);
                if (half == 0) {
                    lo0 = lo;
                    hi0 = hi;
                } else {
                    lo1 = lo;
                    hi1 = hi;
                }
                const E* q = static_cast<const E*>(a.q) + static_cast<int64_t>(rq.row0 + tok) * a.qs[0] +
                             static_cast<int64_t>(hk * a.G + (there ? ri - tok * a.G : 0)) * a.qs[1];
                float v[DP / 16][4];
                float top = 0.f;
#pragma unroll
                for (int s = 0; s < DP / 16; ++s) {
                    const int c = (s >> 2) * 64 + 16 * j + 4 * (s & 3);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        v[s][e] = there && c + e < a.d ? ld_q(q + c + e) : 0.f;
                        top = fmaxf(top, fabsf(v[s][e]));
                    }
                }
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // largest value into [2^7, 2^8); 0 and values that are not finite stay as they are
                const int e = top > 0.f && top < INFINITY ? static_cast<int>(__float_as_uint(top) >> 23) - 127 - 7 : 0;
                const float up = __uint_as_float(static_cast<uint32_t>(127 - min(max(e, -126), 126)) << 23);
                fac[half] = __uint_as_float(static_cast<uint32_t>(127 + min(max(e, -126), 126)) << 23) * a.scale * kLog2e;
#pragma unroll
                for (int s = 0; s < DP / 16; ++s) {
                    const float x0 = v[s][0] * up, x1 = v[s][1] * up, x2 = v[s][2] * up, x3 = v[s][3] * up;
                    const uint32_t p0 = h2(x0, x1), p1 = h2(x2, x3);
                    if constexpr (C::Q_REGS) {
                        qf[s][half] = p0;
                        qf[s][2 + half] = p1;
                    } else {
                        const uint32_t at = my_q + s * 512 * (SPLIT ? 2 : 1) + half * 4;
                        st_shared_u32(at, p0);
                        st_shared_u32(at + 8, p1);
                        if (SPLIT) {
                            const float2 y0 = h2f(p0), y1 = h2f(p1);
                            st_shared_u32(at + 512, h2(x0 - y0.x, x1 - y0.y));
                            st_shared_u32(at + 520, h2(x2 - y1.x, x3 - y1.y));
                        }
                    }
                }
            }
            f0 = fac[0];
            f1 = fac[1];
            in_lo = max(lo0, lo1);                 // keys that no row masks, keys that some row allows
            in_hi = min(hi0, hi1);
            any_lo = min(lo0, lo1);
            any_hi = max(hi0, hi1);
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                in_lo = max(in_lo, __shfl_xor_sync(0xffffffffu, in_lo, o));
                in_hi = min(in_hi, __shfl_xor_sync(0xffffffffu, in_hi, o));
                any_lo = min(any_lo, __shfl_xor_sync(0xffffffffu, any_lo, o));
                any_hi = max(any_hi, __shfl_xor_sync(0xffffffffu, any_hi, o));
            }
            any_hi = min(any_hi, len - 1);
            in_hi = min(in_hi, len - 1);
            if (mt->i0 + rt * 16 >= nr) any_hi = -1;   // no rows at all
            m0 = m1 = M0 = M1 = -INFINITY;
            l0 = l1 = 0.f;
#pragma unroll
            for (int i = 0; i < DVP / 8; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
            __syncwarp();
        }
        const uint32_t kt = sb + stage * C::STAGE, vt = kt + C::K_BYTES;
        for (int ch = slice; ch < 4; ch += slices) {
            const int base = key0 + 16 * ch;
            if (base > any_hi || base + 15 < any_lo) continue;
            // ---- S = Q K^T for 16 keys; n of a fragment is key n (even) or n ^ 4 (odd) of its eight
            const int kr = (g & 1) ? (g ^ 4) : g;
            float s[2][2][4];
#pragma unroll
            for (int i = 0; i < 16; ++i) (&s[0][0][0])[i] = 0.f;
#pragma unroll
            for (int kk = 0; kk < DP / 64; ++kk) {
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const uint4 kv = lds128(kt + (kk >> 1) * kTile * C::RBK +
                                            swz<C::RBK>(16 * ch + 8 * nt + kr, (kk & 1) * 64 + 16 * j));
                    const uint32_t word[4] = {kv.x, kv.y, kv.z, kv.w};
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const uint32_t b0 = cvt2(word[u]), b1 = cvt2_hi(word[u]);
                        if constexpr (C::Q_REGS) {
                            mma(s[nt][u & 1], qf[kk * 4 + u], b0, b1);
                        } else {
                            const uint32_t at = my_q + (kk * 4 + u) * 512 * (SPLIT ? 2 : 1);
                            const uint4 qa = lds128(at);
                            const uint32_t fa[4] = {qa.x, qa.y, qa.z, qa.w};
                            mma(s[nt][u & 1], fa, b0, b1);
                            if (SPLIT) {
                                const uint4 qb = lds128(at + 512);
                                const uint32_t fb[4] = {qb.x, qb.y, qb.z, qb.w};
                                mma(s[nt][u & 1], fb, b0, b1);
                            }
                        }
                    }
                }
            }
            // ---- scores, maxima
            const float ks = mt->ks[ch], vs = mt->vs[ch];
            const float a0 = f0 * ks, a1 = f1 * ks;
            float z[2][4];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
                z[nt][0] = (s[nt][0][0] + s[nt][1][0]) * a0;
                z[nt][1] = (s[nt][0][1] + s[nt][1][1]) * a0;
                z[nt][2] = (s[nt][0][2] + s[nt][1][2]) * a1;
                z[nt][3] = (s[nt][0][3] + s[nt][1][3]) * a1;
            }
            if (base < in_lo || base + 15 > in_hi) {
#pragma unroll
                for (int nt = 0; nt < 2; ++nt) {
                    const int ka = base + 8 * nt + 2 * j, kb = base + 8 * nt + ((2 * j + 1) ^ 4);
                    const bool la = ka >= len, lb = kb >= len;
                    if (la || ka < lo0 || ka > hi0) z[nt][0] = -INFINITY;
                    if (lb || kb < lo0 || kb > hi0) z[nt][1] = -INFINITY;
                    if (la || ka < lo1 || ka > hi1) z[nt][2] = -INFINITY;
                    if (lb || kb < lo1 || kb > hi1) z[nt][3] = -INFINITY;
                }
            }
            float c0 = fmaxf(fmaxf(z[0][0], z[0][1]), fmaxf(z[1][0], z[1][1]));
            float c1 = fmaxf(fmaxf(z[0][2], z[0][3]), fmaxf(z[1][2], z[1][3]));
            c0 = fmaxf(c0, __shfl_xor_sync(0xffffffffu, c0, 1));
            c1 = fmaxf(c1, __shfl_xor_sync(0xffffffffu, c1, 1));
            c0 = fmaxf(c0, __shfl_xor_sync(0xffffffffu, c0, 2));
            c1 = fmaxf(c1, __shfl_xor_sync(0xffffffffu, c1, 2));
            // ---- m, l
            const float n0 = fmaxf(m0, c0), n1 = fmaxf(m1, c1);
            const float e0 = n0 == -INFINITY ? 0.f : n0, e1 = n1 == -INFINITY ? 0.f : n1;
            l0 = l0 * ex2(m0 - e0) + ((ex2(z[0][0] - e0) + ex2(z[0][1] - e0)) + (ex2(z[1][0] - e0) + ex2(z[1][1] - e0)));
            l1 = l1 * ex2(m1 - e1) + ((ex2(z[0][2] - e1) + ex2(z[0][3] - e1)) + (ex2(z[1][2] - e1) + ex2(z[1][3] - e1)));
            m0 = n0;
            m1 = n1;
            if (!(vs > 0.f)) continue;             // a page of zeros: nothing to add (its scale is 0)
            // ---- weights in fp16, relative to M
            const float lv = __log2f(vs), u0 = c0 + lv, u1 = c1 + lv;
            if (__any_sync(0xffffffffu, u0 > M0 + kLazy || u1 > M1 + kLazy)) {
                const float N0 = fmaxf(M0, u0), N1 = fmaxf(M1, u1);
                const float x0 = M0 == -INFINITY ? 0.f : ex2(M0 - N0), x1 = M1 == -INFINITY ? 0.f : ex2(M1 - N1);
#pragma unroll
                for (int i = 0; i < DVP / 8; ++i) {
                    acc[i][0] *= x0;
                    acc[i][1] *= x0;
                    acc[i][2] *= x1;
                    acc[i][3] *= x1;
                }
                M0 = N0;
                M1 = N1;
            }
            const float t0 = (M0 == -INFINITY ? 0.f : M0 - lv) - kOff, t1 = (M1 == -INFINITY ? 0.f : M1 - lv) - kOff;
            uint32_t wf[4], wl[4];
#pragma unroll
            for (int nt = 0; nt < 2; ++nt) {
                const float y0 = ex2(z[nt][0] - t0), y1 = ex2(z[nt][1] - t0), y2 = ex2(z[nt][2] - t1),
                            y3 = ex2(z[nt][3] - t1);
                wf[2 * nt] = h2(y0, y1);
                wf[2 * nt + 1] = h2(y2, y3);
                if (SPLIT) {
                    const float2 r0 = h2f(wf[2 * nt]), r1 = h2f(wf[2 * nt + 1]);
                    wl[2 * nt] = h2(y0 - r0.x, y1 - r0.y);
                    wl[2 * nt + 1] = h2(y2 - r1.x, y3 - r1.y);
                }
            }
            // ---- O += W V: this lane's four keys, CV consecutive channels
            constexpr int CV = (DVP < 128 ? DVP : 128) / 8;          // 8 or 16
            const int key[4] = {2 * j, (2 * j + 1) ^ 4, 8 + 2 * j, 8 + ((2 * j + 1) ^ 4)};
#pragma unroll
            for (int hv = 0; hv < C::HV; ++hv) {
                uint32_t v[4][CV / 4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t at = vt + hv * kTile * C::RBV + swz<C::RBV>(16 * ch + key[i], CV * g);
                    if constexpr (CV == 16) {
                        const uint4 x4 = lds128(at);
                        v[i][0] = x4.x;
                        v[i][1] = x4.y;
                        v[i][2] = x4.z;
                        v[i][3] = x4.w;
                    } else {
                        const uint2 x2 = lds64(at);
                        v[i][0] = x2.x;
                        v[i][1] = x2.y;
                    }
                    // slots past the last token may hold anything: their weight is 0, NaN is not
                    if (base + 16 > len && base + key[i] >= len)
#pragma unroll
                        for (int c = 0; c < CV / 4; ++c) v[i][c] = 0;
                }
#pragma unroll
                for (int c = 0; c < CV / 4; ++c) {
                    const uint32_t ab0 = __byte_perm(v[0][c], v[1][c], 0x5140), ab1 = __byte_perm(v[0][c], v[1][c], 0x7362);
                    const uint32_t cd0 = __byte_perm(v[2][c], v[3][c], 0x5140), cd1 = __byte_perm(v[2][c], v[3][c], 0x7362);
                    const uint32_t b0[4] = {cvt2(ab0), cvt2_hi(ab0), cvt2(ab1), cvt2_hi(ab1)};
                    const uint32_t b1[4] = {cvt2(cd0), cvt2_hi(cd0), cvt2(cd1), cvt2_hi(cd1)};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        mma(acc[hv * CV + 4 * c + e], wf, b0[e], b1[e]);
                        if (SPLIT) mma(acc[hv * CV + 4 * c + e], wl, b0[e], b1[e]);
                    }
                }
            }
        }
        const int row0 = mt->row0, hk = mt->hk, i0 = mt->i0, nr = mt->n * a.G;
        __syncwarp();
        if (lane == 0) mbar_arrive(EMPTY(stage));
        if (++stage == C::NS) {
            stage = 0;
            phase ^= 1;
        }
        if (!(flags & F_LAST)) continue;

        // ---- the end of this CTA's share of the item: join the warps' slices, in a fixed order
        l0 += __shfl_xor_sync(0xffffffffu, l0, 1);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 1);
        l0 += __shfl_xor_sync(0xffffffffu, l0, 2);
        l1 += __shfl_xor_sync(0xffffffffu, l1, 2);
        for (int st = slices >> 1; st >= 1; st >>= 1) {
            float* buf = merge + ((slice & (st - 1)) * w.RT + rt) * (16 * DVP + 64);
            if (slice >= st && slice < 2 * st) {
#pragma unroll
                for (int i = 0; i < DVP / 8; ++i)
                    *reinterpret_cast<float4*>(buf + (i * 32 + lane) * 4) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
                if (j == 0) {
                    float* e = buf + 16 * DVP + g * 8;
                    e[0] = m0;
                    e[1] = l0;
                    e[2] = M0;
                    e[3] = m1;
                    e[4] = l1;
                    e[5] = M1;
                }
            }
            if (!consumers_meet()) return;
            if (slice < st) {
                const float* e = buf + 16 * DVP + g * 8;
                const float bm0 = e[0], bl0 = e[1], bM0 = e[2], bm1 = e[3], bl1 = e[4], bM1 = e[5];
                const float n0 = fmaxf(m0, bm0), n1 = fmaxf(m1, bm1);
                if (n0 != -INFINITY) l0 = l0 * ex2(m0 - n0) + bl0 * ex2(bm0 - n0);
                else l0 += bl0;
                if (n1 != -INFINITY) l1 = l1 * ex2(m1 - n1) + bl1 * ex2(bm1 - n1);
                else l1 += bl1;
                m0 = n0;
                m1 = n1;
                const float N0 = fmaxf(M0, bM0), N1 = fmaxf(M1, bM1);
                const float x0 = M0 == -INFINITY ? 0.f : ex2(M0 - N0), x1 = M1 == -INFINITY ? 0.f : ex2(M1 - N1);
                const float y0 = bM0 == -INFINITY ? 0.f : ex2(bM0 - N0), y1 = bM1 == -INFINITY ? 0.f : ex2(bM1 - N1);
#pragma unroll
                for (int i = 0; i < DVP / 8; ++i) {
                    const float4 v = *reinterpret_cast<const float4*>(buf + (i * 32 + lane) * 4);
                    acc[i][0] = acc[i][0] * x0 + v.x * y0;
                    acc[i][1] = acc[i][1] * x0 + v.y * y0;
                    acc[i][2] = acc[i][2] * x1 + v.z * y1;
                    acc[i][3] = acc[i][3] * x1 + v.w * y1;
                }
                M0 = N0;
                M1 = N1;
            }
            if (!consumers_meet()) return;
        }
        if (slice) continue;
        constexpr int CV = (DVP < 128 ? DVP : 128) / 8;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            const int row = rt * 16 + g + 8 * half, ri = i0 + row;
            if (ri >= nr) continue;
            float m = half ? m1 : m0, l = half ? l1 : l0;
            const float M = half ? M1 : M0;
            if (flags & (F_LEAD | F_TRAIL)) {
                const int64_t slot = (2 * static_cast<int64_t>(cta) + (flags & F_TRAIL ? 1 : 0)) * rows_per + row;
                const float f = M == -INFINITY ? 0.f : ex2(M - kOff - (m == -INFINITY ? 0.f : m));
                if (j == 0) w.ml[slot] = make_float2(m, l);
#pragma unroll
                for (int hv = 0; hv < C::HV; ++hv)
#pragma unroll
                    for (int n = 0; n < 2; ++n) {
                        float* o = w.part + slot * DVP + hv * 128 + CV * (2 * j + n);
#pragma unroll
                        for (int c = 0; c < CV; c += 4)
                            *reinterpret_cast<float4*>(o + c) =
                                make_float4(acc[hv * CV + c][2 * half + n] * f, acc[hv * CV + c + 1][2 * half + n] * f,
                                            acc[hv * CV + c + 2][2 * half + n] * f, acc[hv * CV + c + 3][2 * half + n] * f);
                    }
                continue;
            }
            const int tok = ri / a.G, head = hk * a.G + ri - tok * a.G;
            if (a.sink) {
                const float sk = __ldg(a.sink + head) * kLog2e, nm = fmaxf(m, sk);
                l = (m == -INFINITY ? l : l * ex2(m - nm)) + ex2(sk - nm);
                m = nm;
            }
            if (a.m && j == 0) {
                a.m[static_cast<int64_t>(head) * a.T + row0 + tok] = m == -INFINITY ? m : m * kLn2;
                a.l[static_cast<int64_t>(head) * a.T + row0 + tok] = l;
            }
            const float f = l == 0.f || M == -INFINITY ? (l != l ? l : 0.f) : ex2(M - kOff - m) / l;
            E* o = static_cast<E*>(a.o) + static_cast<int64_t>(row0 + tok) * a.os[0] + static_cast<int64_t>(head) * a.os[1];
#pragma unroll
            for (int hv = 0; hv < C::HV; ++hv)
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const int c0 = hv * 128 + CV * (2 * j + n);
                    if constexpr (!SPLIT) {
                        if (w.vec_o && c0 + CV <= a.dv) {
#pragma unroll
                            for (int c = 0; c < CV; c += 8) {
                                uint32_t p[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    p[e] = pack_bf16(acc[hv * CV + c + 2 * e][2 * half + n] * f, acc[hv * CV + c + 2 * e + 1][2 * half + n] * f);
                                *reinterpret_cast<uint4*>(o + c0 + c) = make_uint4(p[0], p[1], p[2], p[3]);
                            }
                            continue;
                        }
                    }
#pragma unroll
                    for (int c = 0; c < CV; ++c)
                        if (c0 + c < a.dv) o[c0 + c] = static_cast<E>(acc[hv * CV + c][2 * half + n] * f);
                }
        }
    }
}

// Joins the pieces of the items that CTA boundaries cut: the block of the CTA in which an item
// begins, rpb rows of it (a warp per row and every (8 / rpb)-th piece), pieces in ascending order.
template <int DVP, typename E>
__global__ void __launch_bounds__(256) k_cache_join(const Work w, int rpb, uint32_t* out_status) {
    constexpr int V = DVP / 32;
    __shared__ float s_acc[8][DVP];
    __shared__ uint32_t s_flags, s_where;
    const CacheAttnArgs& a = w.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (c == 0 && blockIdx.y == 0) {               // the call's status word
        if (threadIdx.x == 0) s_flags = s_where = 0;
        __syncthreads();
        for (int i = threadIdx.x; i < w.ctas; i += 256)
            if (w.recs[i].flags) {
                atomicOr(&s_flags, w.recs[i].flags);
                atomicMax(&s_where, w.recs[i].where);
            }
        __syncthreads();
        if (threadIdx.x == 0) {
            out_status[0] = s_flags;
            out_status[1] = s_where;
        }
    }
    const Rec rec = w.recs[c];
    const int row = blockIdx.y * rpb + warp % rpb, part = warp / rpb, parts = 8 / rpb;
    if (!rec.trail || static_cast<int>(blockIdx.y) * rpb >= rec.nrows) return;
    int n = 1;                                     // pieces
    for (;;) {
        const int i = c + n + lane;
        const unsigned b = __ballot_sync(0xffffffffu, i >= w.ctas || !w.recs[i].lead || w.recs[i].lead_ends);
        if (b) {
            n += __ffs(b);
            break;
        }
        n += 32;
    }
    n = min(n, w.ctas - c);
    const bool there = row < rec.nrows;
    auto slot = [&](int k) { return (k ? 2 * (static_cast<int64_t>(c) + k) : 2 * static_cast<int64_t>(c) + 1) * (16 * w.RT) + row; };
    float m = -INFINITY, l = 0.f, acc[V];
    if (there)
        for (int k = lane; k < n; k += 32) m = fmaxf(m, w.ml[slot(k)].x);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const float ref = m == -INFINITY ? 0.f : m;
    if (there)
        for (int k = lane; k < n; k += 32) {
            const float2 x = w.ml[slot(k)];
            l += x.y == 0.f ? 0.f : x.y * ex2(x.x - ref);
        }
#pragma unroll
    for (int o = 16; o; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    if (there) {
#pragma unroll 4
        for (int k = part; k < n; k += parts) {
            const int64_t s = slot(k);
            const float2 x = w.ml[s];
            const float f = x.y == 0.f ? 0.f : ex2(x.x - ref);
            const float* p = w.part + s * DVP + lane * V;
            float v[V];
            if constexpr (V == 2) {
                const float2 t = *reinterpret_cast<const float2*>(p);
                v[0] = t.x;
                v[1] = t.y;
            } else {
#pragma unroll
                for (int i = 0; i < V; i += 4) {
                    const float4 t = *reinterpret_cast<const float4*>(p + i);
                    v[i] = t.x;
                    v[i + 1] = t.y;
                    v[i + 2] = t.z;
                    v[i + 3] = t.w;
                }
            }
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = fmaf(f, v[i], acc[i]);
        }
    }
    if (parts > 1) {
        if (part)
#pragma unroll
            for (int i = 0; i < V; ++i) s_acc[warp][lane * V + i] = acc[i];
        __syncthreads();
        if (part) return;
        for (int q = 1; q < parts; ++q)
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] += s_acc[q * rpb + warp][lane * V + i];
    }
    if (!there) return;
    const int ri = rec.i0 + row, tok = ri / a.G, head = rec.hk * a.G + ri - tok * a.G;
    float x = 1.f;
    if (a.sink) {
        const float sk = __ldg(a.sink + head) * kLog2e, nm = fmaxf(m, sk);
        x = m == -INFINITY ? 1.f : ex2(m - nm);
        l = l * x + ex2(sk - nm);
        m = nm;
    }
    if (a.m && lane == 0) {
        a.m[static_cast<int64_t>(head) * a.T + rec.row0 + tok] = m == -INFINITY ? m : m * kLn2;
        a.l[static_cast<int64_t>(head) * a.T + rec.row0 + tok] = l;
    }
    const float f = l == 0.f ? 0.f : x / l;
    E* o = static_cast<E*>(a.o) + static_cast<int64_t>(rec.row0 + tok) * a.os[0] + static_cast<int64_t>(head) * a.os[1];
#pragma unroll
    for (int i = 0; i < V; ++i)
        if (lane * V + i < a.dv) o[lane * V + i] = static_cast<E>(acc[i] * f);
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

constexpr int kMaxSms = 160;          // the workspace is sized for this many

struct Plan {
    int DP, DVP, RT, occ, max_ctas;
    size_t recs, ml, part, total;     // offsets behind the header
};
bool plan_of(const CacheAttnArgs& a, Plan& p) {
    if (a.d % 16 || a.dv % 16 || a.d > 256 || a.dv > 256) return false;
    if (a.P % 16 || (a.P < kTile ? kTile % a.P : a.P % kTile)) return false;
    p.DP = a.d <= 64 ? 64 : a.d <= 128 ? 128 : 256;
    p.DVP = a.dv <= 64 ? 64 : a.dv <= 128 ? 128 : 256;
    if (p.DVP > p.DP) p.DP = p.DVP;
    if (p.DP == 256 && p.DVP == 64) p.DVP = 128;
    const int64_t rows = static_cast<int64_t>(a.max_q > 0 ? a.max_q : 1) * a.G;
    p.RT = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
    p.occ = p.DP <= 128 ? 2 : 1;
    p.max_ctas = kMaxSms * p.occ;
    auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
    const size_t slots = 2 * static_cast<size_t>(p.max_ctas) * 16 * p.RT;
    p.recs = 256;
    p.ml = p.recs + up(sizeof(Rec) * p.max_ctas);
    p.part = p.ml + up(slots * sizeof(float2));
    p.total = p.part + up(slots * p.DVP * sizeof(float));
    return true;
}

template <int DP, int DVP, bool SPLIT>
cudaError_t launch(const Work& w, const CUtensorMap* maps, int rpb, cudaStream_t s) {
    using C = Cfg<DP, DVP, SPLIT>;
    auto kernel = k_cache_attn_mma<DP, DVP, SPLIT>;
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t{1} << (dev & 63);
    if (!(done.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::smem(4));
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    kernel<<<w.ctas, kThreads, C::smem(w.RT), s>>>(maps[0], maps[1], w);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(w.ctas, 16 * w.RT / rpb);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    using E = typename std::conditional<SPLIT, float, __nv_bfloat16>::type;
    return cudaLaunchKernelEx(&cfg, k_cache_join<DVP, E>, w, rpb, w.a.status);
}

}  // namespace

bool cache_attn_mma_supported(const CacheAttnArgs& a) {
    Plan p;
    return plan_of(a, p);
}

size_t cache_attn_mma_workspace(const CacheAttnArgs& a) {
    Plan p;
    return plan_of(a, p) ? p.total : 256;
}

CacheBox cache_attn_mma_box(const CacheAttnArgs& a) {
    Plan p;
    plan_of(a, p);
    return {p.DP < 128 ? p.DP : 128, p.DVP < 128 ? p.DVP : 128, a.P < kTile ? a.P : kTile};
}

cudaError_t launch_cache_attn_mma(const CacheAttnArgs& a, const CUtensorMap* maps, uint8_t* ws, cudaStream_t s) {
    Plan p;
    if (!plan_of(a, p)) return cudaErrorInvalidValue;
    Work w;
    w.a = a;
    w.RT = p.RT;
    // no more CTAs than the longest table rows have tiles
    const int64_t groups = (static_cast<int64_t>(a.max_q > 0 ? a.max_q : 1) * a.G + 16 * p.RT - 1) / (16 * p.RT);
    const int64_t most = ((static_cast<int64_t>(a.max_pages) * a.P + kTile - 1) / kTile) * a.Hkv * a.R * groups;
    const int64_t ctas = static_cast<int64_t>(std::min(sm_count(), kMaxSms)) * p.occ;
    w.ctas = static_cast<int>(most < ctas ? most : ctas);
    w.recs = reinterpret_cast<Rec*>(ws + p.recs);
    w.ml = reinterpret_cast<float2*>(ws + p.ml);
    w.part = reinterpret_cast<float*>(ws + p.part);
    w.vec_o = a.dtype == BPA_BF16 && (reinterpret_cast<uintptr_t>(a.o) & 15) == 0 && a.os[0] % 8 == 0 && a.os[1] % 8 == 0;
    // rows of a join block: few when an item is cut into many pieces
    const int64_t pieces = w.ctas / (static_cast<int64_t>(a.R) * a.Hkv);
    const int rpb = pieces <= 4 ? 8 : pieces <= 16 ? 4 : pieces <= 64 ? 2 : 1;
    const bool f32 = a.dtype == BPA_FP32;
#define BPA_CACHE_CASE(DP_, DVP_) \
    if (p.DP == DP_ && p.DVP == DVP_) \
        return f32 ? launch<DP_, DVP_, true>(w, maps, rpb, s) : launch<DP_, DVP_, false>(w, maps, rpb, s);
    BPA_CACHE_CASE(64, 64)
    BPA_CACHE_CASE(128, 64)
    BPA_CACHE_CASE(128, 128)
    BPA_CACHE_CASE(256, 128)
    BPA_CACHE_CASE(256, 256)
#undef BPA_CACHE_CASE
    return cudaErrorInvalidValue;
}

}  // namespace bpa
