// cache_attn_tc.cu - attention of many query rows over the paged 8-bit cache (prompts, pieces of
// prompts) on the 5th-generation tensor cores.  bf16 rows, head dims up to 128.
//
// An item is 256 query rows (row = token-in-request * G + q head in the group: they read the same
// keys) of one request and kv head, as two tiles of 128 rows; persistent CTAs, one per SM, take items
// from a counter and walk their keys in tiles of 128.  e4m3 codes are exact in fp16, so K and V
// are only converted (one instruction for two codes) and the pages' scales are applied in float32:
//   S = Q K^T     Q scaled by a power of two per row into fp16's range;
//   x = S * (k scale * row's scale * softmax scale), log2 units;  u = x + log2(v scale)
//   W = exp2(u - M + 7) in fp16, M the row's running maximum of u (moved only when it grows by
//       more than 8, so W <= 2^15);  O += W V;  L += sum W / (v scale);  o = O / L
// One exponential serves the numerator and the denominator, with 1 / (v scale) relative to the first
// scale that the item meets; a page below 2^-100 of that one, or of zeros (scale 0), counts as 2^-100 of it.
//
// Bounded by the softmax's instructions and the exponentials beside the products (compute, not
// bytes): per 128 x 128 scores of one row tile a thread owns a row and spends about three instructions
// and one exponential a score.
// Roles (512 threads; registers moved to the softmax by setmaxnreg):
//   warps 0-3, 4-7   softmax of tile 0, 1; they also bring their rows of Q into shared memory
//   warp 8           MMA issuer, TMEM owner
//   warp 9           items, and for each key tile its pages' ids and scales (a ring of records)
//   warps 12-15      K and V: global memory -> registers (one tile ahead) -> fp16 -> swizzled tiles
// TMEM: S0 [0,128), S1 [128,256), O0 [256,256+DV), O1 [384,384+DV); W over the first half of S.
// Every wait is bounded; on a timeout the roles leave their loops and the CTA frees its TMEM.
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>

#include "cache.h"
#include "common.cuh"

namespace bpa {
namespace {

constexpr int kThreads = 512;
constexpr int BN = 128;               // keys of a tile
constexpr int kRows = 256;            // rows of an item
constexpr int kMetas = 4;             // records of key tiles in flight
constexpr float kTau = 8.f, kOff = 7.f;
constexpr float kFar = 100.f;         // log2 of the largest ratio of the v scales below the item's first

struct TileMeta {
    int64_t k[8], v[8];               // where each 16 keys begin in k_cache, v_cache (-1: no page)
    int key0, len, end, pad;
    float a[8], lv[8], e[8];          // k scale * softmax scale * log2(e); log2 v scale; 2^(lv0 - lv)
};
struct Item {
    int valid, row0, n, len, hk, i0, first, tiles;   // first key tile, tiles
    float lv0;
    int pad[3];
};

template <int D, int DV>
struct Cfg {
    static constexpr int SUB = 128 * 128;                        // a slab of 64 fp16 columns x 128 rows
    static constexpr int Q_BYTES = D / 64 * SUB, K_BYTES = D / 64 * SUB, V_BYTES = DV / 64 * SUB;
    static constexpr int NS = 2;
    static constexpr int OFF_K = 2 * Q_BYTES, OFF_V = OFF_K + NS * K_BYTES, OFF_META = OFF_V + NS * V_BYTES;
    static constexpr int OFF_ITEM = OFF_META + kMetas * (int)sizeof(TileMeta), OFF_BAR = OFF_ITEM + 2 * (int)sizeof(Item);
    static constexpr int B_Q = 0, B_KF = 2, B_KE = B_KF + NS, B_VF = B_KE + NS, B_VE = B_VF + NS, B_S = B_VE + NS,
                         B_P = B_S + 2, B_O = B_P + 2, B_OE = B_O + 2, B_MF = B_OE + 2, B_ME = B_MF + kMetas,
                         B_IF = B_ME + kMetas, B_IE = B_IF + 2, B_FIN = B_IE + 2, NBAR = B_FIN + 1;
    static constexpr int SMEM = 1024 + OFF_BAR + 8 * NBAR + 16;
    static_assert(SMEM <= 232448, "shared memory");
    static constexpr uint32_t F16 = 1u << 4;                     // float32 sums, both operands fp16
    static constexpr uint32_t IDESC_S = F16 | (BN >> 3) << 17 | (128 >> 4) << 24;
    static constexpr uint32_t IDESC_PV = F16 | 1u << 16 | (DV >> 3) << 17 | (128 >> 4) << 24;   // V: MN-major
};

// A request's items: nothing for one that the kernel for few rows takes.
BPA_DEV int groups_of(const CacheAttnArgs& a, const Req& q) {
    const int rows = q.n * a.G;
    return rows > kFewRows ? (rows + kRows - 1) / kRows : 0;
}

BPA_DEV uint32_t h2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
BPA_DEV uint32_t cvt_lo(uint32_t four) {   // codes 0, 1 of four -> fp16 pair
    uint32_t h;
    asm("{.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;}" : "=r"(h) : "r"(four));
    return h;
}
BPA_DEV uint32_t cvt_hi(uint32_t four) {
    uint32_t h;
    asm("{.reg .b16 l, u;\n\tmov.b32 {l, u}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, u;}" : "=r"(h) : "r"(four));
    return h;
}

// One pass over the row's 128 scores: weights (fp16 pairs), the row's sum of W e, and the maxima of u
// and x.  EDGE: keys outside [kmin, kmax] are masked.
template <bool EDGE>
BPA_DEV void pass(uint32_t tS, const TileMeta* mt, float f_row, float mref, int k0, int kmin, int kmax, uint32_t (&pk)[64],
                  float& sum, float& umax, float& xmax) {
    sum = 0.f;
    umax = xmax = -INFINITY;
#pragma unroll
    for (int cc = 0; cc < 4; ++cc) {
        uint32_t s[32];
        tmem_ld32(tS + cc * 32, s);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int ch = 2 * cc + h;
            const float a = f_row * mt->a[ch], lv = mt->lv[ch], b = lv - mref;
            const uint64_t a2 = f2_pack(a, a), b2 = f2_pack(b, b);
            uint64_t r2 = 0;
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float s0 = __uint_as_float(s[16 * h + 2 * i]), s1 = __uint_as_float(s[16 * h + 2 * i + 1]);
                float y0, y1;
                if (EDGE) {
                    const int k = k0 + 16 * ch + 2 * i;
                    y0 = k < kmin || k > kmax ? -INFINITY : s0 * a;
                    y1 = k + 1 < kmin || k + 1 > kmax ? -INFINITY : s1 * a;
                    mx = fmax3(mx, y0, y1);
                    y0 += b;
                    y1 += b;
                } else {
                    mx = fmax3(mx, s0, s1);
                    f2_unpack(ffma2(f2_pack(s0, s1), a2, b2), y0, y1);
                }
                const float w0 = ex2(y0), w1 = ex2(y1);
                r2 = fadd2(r2, f2_pack(w0, w1));
                pk[8 * ch + i] = h2(w0, w1);
            }
            const float x = EDGE ? mx : mx * a;                   // a >= 0
            umax = fmaxf(umax, x + lv);
            xmax = fmaxf(xmax, x);
            float p, q;
            f2_unpack(r2, p, q);
            sum = fmaf(p + q, mt->e[ch], sum);
        }
    }
}

template <int D, int DV>
__global__ void __launch_bounds__(kThreads, 1) k_cache_attn_tc(const CacheAttnArgs a, uint32_t* counter, int vec_q, int vec_o) {
    using C = Cfg<D, DV>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
    const uint32_t sb = smem_u32(smem), bar0 = sb + C::OFF_BAR;
    auto BAR = [&](int i) { return bar0 + 8u * i; };
    TileMeta* metas = reinterpret_cast<TileMeta*>(smem + C::OFF_META);
    Item* items = reinterpret_cast<Item*>(smem + C::OFF_ITEM);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + 8 * C::NBAR);
    volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(BAR(C::B_Q + i), 128);
            mbar_init(BAR(C::B_S + i), 1);
            mbar_init(BAR(C::B_P + i), 128);
            mbar_init(BAR(C::B_O + i), 1);
            mbar_init(BAR(C::B_OE + i), 128);
            mbar_init(BAR(C::B_IF + i), 1);
            mbar_init(BAR(C::B_IE + i), 9);        // MMA warp, eight softmax warps
        }
        for (int i = 0; i < C::NS; ++i) {
            mbar_init(BAR(C::B_KF + i), 4);
            mbar_init(BAR(C::B_KE + i), 1);
            mbar_init(BAR(C::B_VF + i), 4);
            mbar_init(BAR(C::B_VE + i), 1);
        }
        for (int i = 0; i < kMetas; ++i) {
            mbar_init(BAR(C::B_MF + i), 1);
            mbar_init(BAR(C::B_ME + i), 12);       // four converting and eight softmax warps
        }
        mbar_init(BAR(C::B_FIN), 1);
        *abort = 0;
        fence_mbar_init();
    }
    if (warp == 8) {
        tmem_alloc(smem_u32(tmem_slot), 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    auto wait = [&](int b, int parity, uint32_t where) {
        return __all_sync(0xffffffffu, mbar_wait(BAR(b), parity & 1, abort, a.status, where)) != 0;
    };

    if (warp >= 12) {
        // ------------------------------------------------------------ K, V: codes -> fp16 tiles
        asm volatile("setmaxnreg.dec.sync.aligned.u32 96;");
        const int wq = warp - 12, c = lane & 7, r4 = lane >> 3;        // 16-byte piece of a row; row of four
        uint4 kr[8], vr[8];
        // this thread's pieces of a tile: rows 32 wq + 4 i + r4, so two stretches of 16 keys
        auto load = [&](const TileMeta* mt, const int64_t* starts, const uint8_t* base, int64_t step, int ch, uint4 (&x)[8]) {
            const int left = mt->len - mt->key0 - 32 * wq - r4;        // rows of this thread that are keys: 4 i < left
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int64_t at = starts[2 * wq + h];
                const uint8_t* p = base + at + r4 * step + 16 * c;
                const bool some = at >= 0 && 16 * c < ch;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[4 * h + i] = make_uint4(0, 0, 0, 0);
                    if (some && 16 * h + 4 * i < left) x[4 * h + i] = *reinterpret_cast<const uint4*>(p + 4 * i * step);
                }
            }
        };
        auto store = [&](uint8_t* tile, int width, const uint4 (&x)[8]) {
            if (16 * c >= width) return;
            uint8_t* slab = tile + (c >> 2) * C::SUB;
            const int flip = c >> 2;                                   // the halves of a row on other banks
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int row = 32 * wq + 4 * i + r4;
                const uint4 lo = make_uint4(cvt_lo(x[i].x), cvt_hi(x[i].x), cvt_lo(x[i].y), cvt_hi(x[i].y));
                const uint4 hi = make_uint4(cvt_lo(x[i].z), cvt_hi(x[i].z), cvt_lo(x[i].w), cvt_hi(x[i].w));
                *reinterpret_cast<uint4*>(slab + sw128_offset(row, (c & 3) * 2 + flip)) = flip ? hi : lo;
                *reinterpret_cast<uint4*>(slab + sw128_offset(row, (c & 3) * 2 + 1 - flip)) = flip ? lo : hi;
            }
        };
        int t = 0;
        bool ok = wait(C::B_MF, 0, 0xE0);
        bool more = ok && !metas[0].end;
        if (more) {
            load(&metas[0], metas[0].k, a.kc, a.kcs[2], a.d, kr);
            load(&metas[0], metas[0].v, a.vc, a.vcs[2], a.dv, vr);
        }
        for (; ok && more; ++t) {
            const int st = t % C::NS, use = t / C::NS;
            const int next = (t + 1) % kMetas;
            if (use > 0 && !(ok = wait(C::B_KE + st, use - 1, 0xE1))) break;
            store(smem + C::OFF_K + st * C::K_BYTES, D, kr);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(C::B_KF + st));
            if (!(ok = wait(C::B_MF + next, (t + 1) / kMetas, 0xE2))) break;
            more = !metas[next].end;
            if (more) load(&metas[next], metas[next].k, a.kc, a.kcs[2], a.d, kr);
            if (use > 0 && !(ok = wait(C::B_VE + st, use - 1, 0xE3))) break;
            store(smem + C::OFF_V + st * C::V_BYTES, DV, vr);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(BAR(C::B_VF + st));
                mbar_arrive(BAR(C::B_ME + t % kMetas));                // its codes have been loaded
            }
            if (more) load(&metas[next], metas[next].v, a.vc, a.vcs[2], a.dv, vr);
        }
    } else if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
        if (warp == 9) {
            // -------------------------------------------------------- items and their key tiles' records
            int t = 0;                 // records written
            auto publish_end = [&]() {
                if (t >= kMetas && !wait(C::B_ME + t % kMetas, t / kMetas - 1, 0xE4)) return;
                if (lane == 0) {
                    metas[t % kMetas].end = 1;
                    mbar_arrive(BAR(C::B_MF + t % kMetas));
                }
            };
            for (int k = 0;; ++k) {
                if (k >= 2 && !wait(C::B_IE + (k & 1), (k >> 1) - 1, 0xE5)) break;
                uint32_t idx = 0;
                if (lane == 0) idx = atomicAdd(counter, 1u);
                idx = __shfl_sync(0xffffffffu, idx, 0);
                // the item's request: a running sum over the requests, 32 at a time
                Req rq = {};
                int r = -1, groups = 0;
                for (int base = 0; base < a.R; base += 32) {
                    Req q = {};
                    if (base + lane < a.R) q = request_of(a, base + lane);
                    const int gr = groups_of(a, q);
                    uint32_t x = static_cast<uint32_t>(gr) * a.Hkv;
                    const uint32_t own = x;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
                        if (lane >= o) x += y;
                    }
                    const unsigned hit = __ballot_sync(0xffffffffu, idx < x);
                    if (hit) {
                        const int src = __ffs(hit) - 1;
                        idx -= __shfl_sync(0xffffffffu, x - own, src);
                        r = base + src;
                        groups = __shfl_sync(0xffffffffu, gr, src);
                        rq.row0 = __shfl_sync(0xffffffffu, q.row0, src);
                        rq.n = __shfl_sync(0xffffffffu, q.n, src);
                        rq.len = __shfl_sync(0xffffffffu, q.len, src);
                        rq.bad = __shfl_sync(0xffffffffu, static_cast<int>(q.bad), src);
                        break;
                    }
                    idx -= __shfl_sync(0xffffffffu, x, 31);
                }
                Item* it = items + (k & 1);
                if (r < 0) {
                    if (lane == 0) {
                        it->valid = 0;
                        mbar_arrive(BAR(C::B_IF + (k & 1)));
                    }
                    break;
                }
                if (rq.bad && lane == 0) report(a.status, ST_CHECK, 0xCE1);
                const int hk = idx % a.Hkv, i0 = (groups - 1 - static_cast<int>(idx / a.Hkv)) * kRows;   // last rows first
                const int last = min(rq.n * a.G, i0 + kRows) - 1;
                int lo, hi, y;
                row_keys(a, rq, i0 / a.G, lo, y);
                row_keys(a, rq, last / a.G, y, hi);
                const int first = lo <= hi ? lo / BN : 0, tiles = lo <= hi ? hi / BN - first + 1 : 0;
                // lanes 0..7: 16 keys each; a tile's page ids are asked for two tiles ahead, its scales one
                const int32_t* table = a.table + static_cast<int64_t>(r) * a.max_pages;
                auto page_of = [&](int j) {
                    const int key = (first + j) * BN + 16 * lane;
                    return lane < 8 && j < tiles && key < rq.len ? table[key / a.P] : INT_MIN;
                };
                auto scales_of = [&](int& id, float& ks, float& vs) {
                    ks = vs = 0.f;
                    if (id >= 0 && id < a.num_pages) {
                        ks = a.kscale[static_cast<int64_t>(id) * a.Hkv + hk];
                        vs = a.vscale[static_cast<int64_t>(id) * a.Hkv + hk];
                    } else {
                        if (id != INT_MIN) report(a.status, ST_CHECK, 0xCE0);
                        id = -1;
                    }
                };
                int id = page_of(0), id1 = page_of(1);
                float ks, vs;
                scales_of(id, ks, vs);
                const unsigned some = __ballot_sync(0xffffffffu, vs > 0.f);
                const float lv0 = some ? __log2f(__shfl_sync(0xffffffffu, vs, __ffs(some) - 1)) : 0.f;
                if (lane == 0) {
                    *it = {1, rq.row0, rq.n, rq.len, hk, i0, first, tiles, lv0, {}};
                    mbar_arrive(BAR(C::B_IF + (k & 1)));
                }
                bool ok = true;
                for (int j = 0; j < tiles; ++j, ++t) {
                    const int sl = t % kMetas, id2 = page_of(j + 2);
                    float ks1, vs1;
                    scales_of(id1, ks1, vs1);
                    if (t >= kMetas && !(ok = wait(C::B_ME + sl, t / kMetas - 1, 0xE6))) break;
                    TileMeta* m = metas + sl;
                    if (lane < 8) {
                        const int tok = ((first + j) * BN + 16 * lane) % a.P;
                        const float lv = vs > 0.f ? fmaxf(__log2f(vs), lv0 - kFar) : lv0 - kFar;
                        m->k[lane] = id < 0 ? -1 : id * a.kcs[0] + hk * a.kcs[1] + tok * a.kcs[2];
                        m->v[lane] = id < 0 ? -1 : id * a.vcs[0] + hk * a.vcs[1] + tok * a.vcs[2];
                        m->a[lane] = ks * a.scale * kLog2e;
                        m->lv[lane] = lv;
                        m->e[lane] = ex2(lv0 - lv);
                    }
                    if (lane == 0) {
                        m->key0 = (first + j) * BN;
                        m->len = rq.len;
                        m->end = 0;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(BAR(C::B_MF + sl));
                    id = id1;
                    ks = ks1;
                    vs = vs1;
                    id1 = id2;
                }
                if (!ok) break;
            }
            publish_end();
        } else if (warp == 8) {
            // -------------------------------------------------------- MMA issuer
            int t = 0, np[2] = {0, 0}, seen[2] = {0, 0};   // key tiles; W tiles used, items with work, per row tile
            bool ok = true;
            for (int k = 0; ok; ++k) {
                if (!wait(C::B_IF + (k & 1), k >> 1, 0xE7)) break;
                const Item it = items[k & 1];
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(C::B_IE + (k & 1)));
                if (!it.valid) break;
                if (it.tiles == 0) continue;
                const int two = it.n * a.G - it.i0 > 128 ? 2 : 1;
                auto issue_s = [&](int i, int pos) {
                    const uint64_t qd = sdesc_sw128(sb + i * C::Q_BYTES, 16, 1024);
                    const uint64_t kd = sdesc_sw128(sb + C::OFF_K + pos % C::NS * C::K_BYTES, 16, 1024);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * C::SUB + (kk & 3) * 32;
                        tc_mma_ss_w(tmem + i * BN, sdesc_advance(qd, off), sdesc_advance(kd, off), C::IDESC_S, kk > 0);
                    }
                    tc_commit_w(BAR(C::B_S + i));
                };
                auto issue_pv = [&](int i, int pos, bool first) {
                    const uint64_t vd = sdesc_sw128(sb + C::OFF_V + pos % C::NS * C::V_BYTES, C::SUB, 1024);
#pragma unroll
                    for (int kk = 0; kk < BN / 16; ++kk)
                        tc_mma_ts_w(tmem + 256 + i * 128, tmem + i * BN + kk * 8, sdesc_advance(vd, kk * 2048), C::IDESC_PV,
                                    (!first || kk > 0) ? 1u : 0u);
                };
                for (int i = 0; ok && i < two; ++i) ok = wait(C::B_Q + i, seen[i], 0xE8);
                ok = ok && wait(C::B_KF + t % C::NS, t / C::NS, 0xE9);
                if (!ok) break;
                tc_fence_after();
                for (int i = 0; i < two; ++i) issue_s(i, t);
                for (int j = 0; ok && j < it.tiles; ++j, ++t) {
                    if (!(ok = wait(C::B_VF + t % C::NS, t / C::NS, 0xEA))) break;
                    for (int i = 0; i < two; ++i) {
                        if (!(ok = wait(C::B_P + i, np[i], 0xEB))) break;
                        // O of the previous item has been read before the first product of this one
                        if (j == 0 && seen[i] > 0 && !(ok = wait(C::B_OE + i, seen[i] - 1, 0xEC))) break;
                        ++np[i];
                        if (i == two - 1) tc_commit_w(BAR(C::B_KE + t % C::NS));   // S(j) is complete
                        tc_fence_after();
                        issue_pv(i, t, j == 0);
                        if (j == it.tiles - 1) tc_commit_w(BAR(C::B_O + i));
                        if (j + 1 < it.tiles) {
                            if (i == 0) {
                                if (!(ok = wait(C::B_KF + (t + 1) % C::NS, (t + 1) / C::NS, 0xED))) break;
                                tc_fence_after();
                            }
                            issue_s(i, t + 1);
                        }
                    }
                    if (!ok) break;
                    tc_commit_w(BAR(C::B_VE + t % C::NS));
                }
                for (int i = 0; i < two; ++i) ++seen[i];
            }
            // every product issued is complete before TMEM is freed
            tc_commit_w(BAR(C::B_FIN));
            int never = 0;
            mbar_wait(BAR(C::B_FIN), 0, &never, a.status, 0xEE);
        }
    } else {
        // ------------------------------------------------------------ softmax: thread t owns row t of its tile
        asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
        const int qt = warp >> 2, row = threadIdx.x & 127;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + qt * BN + lanes, tO = tmem + 256 + qt * 128 + lanes;
        int t = 0, cs = 0, seen = 0;   // key tiles, S tiles and items with work of this row tile
        bool ok = true;
        for (int k = 0; ok; ++k) {
            if (!wait(C::B_IF + (k & 1), k >> 1, 0xF0)) break;
            const Item it = items[k & 1];
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(C::B_IE + (k & 1)));
            if (!it.valid) break;
            const int rows = it.n * a.G, ri = it.i0 + qt * 128 + row;
            const bool there = ri < rows, busy = it.i0 + qt * 128 < rows;     // busy: the tile has rows
            const int tok = there ? ri / a.G : 0, head = it.hk * a.G + (there ? ri - tok * a.G : 0);
            const Req rq = {it.row0, it.n, it.len, false};
            int kmin = 0, kmax = INT_MAX;      // a row that is not there masks nothing (q = 0)
            if (there) row_keys(a, rq, tok, kmin, kmax);
            float f_row = 1.f;
            if (busy && it.tiles) {
                // ---- the row of q as fp16, its largest value scaled into [2^7, 2^8)
                const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + static_cast<int64_t>(it.row0 + tok) * a.qs[0] +
                                         static_cast<int64_t>(head) * a.qs[1];
                uint4 x[D / 8];
                uint32_t top = 0;
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    x[c] = make_uint4(0, 0, 0, 0);
                    if (there && 8 * c < a.d) {
                        if (vec_q) {
                            x[c] = *reinterpret_cast<const uint4*>(q + 8 * c);
                        } else {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const unsigned short* p = reinterpret_cast<const unsigned short*>(q + 8 * c + 2 * e);
                                w[e] = p[0] | static_cast<uint32_t>(p[1]) << 16;
                            }
                            x[c] = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                    const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fff0000u, (w[e] << 16) & 0x7fff0000u));
                }
                int ex = top && top < 0x7f800000u ? static_cast<int>(top >> 23) - 127 - 7 : 0;
                ex = min(max(ex, -126), 126);
                const float up = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
                f_row = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
                uint8_t* tile = smem + qt * C::Q_BYTES;
#pragma unroll
                for (int c = 0; c < D / 8; ++c) {
                    const uint32_t w[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
                    uint32_t y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        y[e] = h2(__uint_as_float(w[e] << 16) * up, __uint_as_float(w[e] & 0xffff0000u) * up);
                    *reinterpret_cast<uint4*>(tile + (c >> 3) * C::SUB + sw128_offset(row, c & 7)) = make_uint4(y[0], y[1], y[2], y[3]);
                }
                fence_proxy_async_smem();
                mbar_arrive(BAR(C::B_Q + qt));
            }
            float M = -INFINITY, xm = -INFINITY, L = 0.f;
            for (int j = 0; j < it.tiles; ++j, ++t) {
                const int sl = t % kMetas, k0 = (it.first + j) * BN;
                if (!busy) {                   // no rows: only the record's turn
                    if (!(ok = wait(C::B_MF + sl, t / kMetas, 0xF1))) break;
                    if (lane == 0) mbar_arrive(BAR(C::B_ME + sl));
                    continue;
                }
                if (!(ok = wait(C::B_MF + sl, t / kMetas, 0xF1) && wait(C::B_S + qt, cs, 0xF2))) break;
                ++cs;
                tc_fence_after();
                const TileMeta* mt = metas + sl;
                const bool edge = __any_sync(0xffffffffu, k0 < kmin || k0 + BN - 1 > kmax);
                uint32_t pk[64];
                float sum, um, x;
                // a second round where a row of the warp moves its M (always for the first tile)
#pragma unroll 1
                for (;;) {
                    const float mref = M == -INFINITY ? 0.f : M - kOff;
                    if (edge) pass<true>(tS, mt, f_row, mref, k0, kmin, kmax, pk, sum, um, x);
                    else pass<false>(tS, mt, f_row, mref, k0, kmin, kmax, pk, sum, um, x);
                    if (!__any_sync(0xffffffffu, um > M + kTau)) break;
                    float fac = 1.f;
                    if (um > M + kTau) {
                        fac = M == -INFINITY ? 0.f : ex2(M - um);
                        M = um;
                        L *= fac;
                    }
                    if (j == 0) continue;
                    // S(j) is complete, so every earlier W V has been added to O
#pragma unroll 1
                    for (int cc = 0; cc < DV / 32; ++cc) {
                        uint32_t r[32];
                        tmem_ld32(tO + cc * 32, r);
#pragma unroll
                        for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * fac);
                        tmem_st32(tO + cc * 32, r);
                    }
                }
                L += sum;
                xm = fmaxf(xm, x);
                tmem_st64(tS, pk);
                tc_fence_before();
                mbar_arrive(BAR(C::B_P + qt));
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(C::B_ME + sl));
            }
            if (!ok) break;
            if (!busy) continue;
            if (it.tiles) {
                if (!(ok = wait(C::B_O + qt, seen, 0xF3))) break;
                tc_fence_after();
                ++seen;
            }
            // ---- epilogue: o = O 2^lv0 / L; l relative to the row's maximum of x
            float l = M == -INFINITY ? (L != L ? L : 0.f) : L * ex2(M - kOff - it.lv0 - xm), mm = xm, share = 1.f;
            if (a.sink) {
                const float sk = __ldg(a.sink + head) * kLog2e, nm = fmaxf(xm, sk);
                const float old = l;
                l = (xm == -INFINITY ? l : l * ex2(xm - nm)) + ex2(sk - nm);
                share = xm == -INFINITY || old == 0.f ? (old != old ? old : 0.f) : old * ex2(xm - nm) / l;   // what the keys have of the row
                mm = nm;
            }
            const float inv = (L == 0.f || M == -INFINITY ? (L != L ? L : 0.f) : ex2(it.lv0) / L) * share;
            const int64_t out_row = it.row0 + tok;
            if (there && a.m) {
                a.m[static_cast<int64_t>(head) * a.T + out_row] = mm == -INFINITY ? mm : mm * kLn2;
                a.l[static_cast<int64_t>(head) * a.T + out_row] = l;
            }
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o) + out_row * a.os[0] + static_cast<int64_t>(head) * a.os[1];
#pragma unroll 1
            for (int cc = 0; cc < DV / 32; ++cc) {
                uint32_t r[32];
                if (it.tiles) {
                    tmem_ld32(tO + cc * 32, r);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; ++i) r[i] = 0;
                }
                if (!there) continue;
#pragma unroll
                for (int v = 0; v < 4; ++v) {
                    if (cc * 32 + 8 * v >= a.dv) continue;
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = pack_bf16(__uint_as_float(r[8 * v + 2 * e]) * inv, __uint_as_float(r[8 * v + 2 * e + 1]) * inv);
                    if (vec_o) {
                        *reinterpret_cast<uint4*>(o + cc * 32 + 8 * v) = make_uint4(w[0], w[1], w[2], w[3]);
                    } else {
                        unsigned short* p = reinterpret_cast<unsigned short*>(o + cc * 32 + 8 * v);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            p[2 * e] = static_cast<unsigned short>(w[e]);
                            p[2 * e + 1] = static_cast<unsigned short>(w[e] >> 16);
                        }
                    }
                }
            }
            if (it.tiles) {
                tc_fence_before();
                mbar_arrive(BAR(C::B_OE + qt));
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, int DV>
cudaError_t launch(const CacheAttnArgs& a, uint32_t* counter, cudaStream_t s) {
    using C = Cfg<D, DV>;
    static std::atomic<int> sms[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    int n = sms[dev & 63].load(std::memory_order_relaxed);
    if (n == 0) {
        if ((e = cudaFuncSetAttribute(k_cache_attn_tc<D, DV>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM)) != cudaSuccess ||
            (e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
            return e;
        sms[dev & 63].store(n, std::memory_order_relaxed);
    }
    const bool vec_q = (reinterpret_cast<uintptr_t>(a.q) & 15) == 0 && a.qs[0] % 8 == 0 && a.qs[1] % 8 == 0;
    const bool vec_o = (reinterpret_cast<uintptr_t>(a.o) & 15) == 0 && a.os[0] % 8 == 0 && a.os[1] % 8 == 0;
    // at most the packed rows' groups and a ragged one per request
    const int64_t most = (static_cast<int64_t>(a.T) * a.G / kRows + a.R) * a.Hkv;
    k_cache_attn_tc<D, DV><<<static_cast<unsigned>(std::min<int64_t>(n, most)), kThreads, C::SMEM, s>>>(a, counter, vec_q, vec_o);
    return cudaGetLastError();
}

}  // namespace

bool cache_attn_tc_supported(const CacheAttnArgs& a) {
    if (a.dtype != BPA_BF16 || a.d % 16 || a.dv % 16 || a.d > 128 || a.dv > 128 || (a.d <= 64 && a.dv > 64) || a.P % 16) return false;
    uintptr_t all = reinterpret_cast<uintptr_t>(a.kc) | reinterpret_cast<uintptr_t>(a.vc);
    for (int i = 0; i < 3; ++i) all |= static_cast<uintptr_t>(a.kcs[i]) | static_cast<uintptr_t>(a.vcs[i]);
    return all % 16 == 0;
}

cudaError_t launch_cache_attn_tc(const CacheAttnArgs& a, uint32_t* counter, cudaStream_t s) {
    if (a.d <= 64) return launch<64, 64>(a, counter, s);
    return a.dv <= 64 ? launch<128, 64>(a, counter, s) : launch<128, 128>(a, counter, s);
}

}  // namespace bpa
