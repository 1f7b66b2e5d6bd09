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
// scale lv0 that the item meets.  That holds while a request's scales lie within a factor 2^40 of it: W
// e = 2^(x + lv0 - M + 7) is then at most 2^75 (2^105 summed over 2^30 keys) and a key of the largest x has W
// >= 2^-93.  A request with a scale outside is marked in `far`, and the kernel for few rows, which has an
// exponential for each of the two sums and takes any scales, computes it again.  Pages of zeros (scale 0)
// have no scale of their own: they count 2^-20 below the largest met so far, so their keys stay in L (far
// below, W would leave float32's range) and do not push the others' W out of fp16's.
//
// Bounded by the softmax's instructions and the exponentials beside the products (compute, not
// bytes): about three instructions and one exponential a score.  Two threads share a row (64 columns
// each), so sixteen warps work on the softmax and cover each other's latencies; its loops stay rolled,
// since unrolled ones kept the warps waiting for instructions.  Five pieces of prompts, 6,852 rows of 32
// heads over up to 16,000 tokens, 128 channels: 1,540 us, 917 TFLOP/s (2,222 us with a thread to a row
// and unrolled loops; 1,738 with eight converting warps; the kernel for few rows 7,225).
// Roles (768 threads; registers moved to the softmax by setmaxnreg):
//   warps 0-7, 8-15  softmax of row tile 0, 1; of eight warps the second four take columns 64-127.  They
//                    also bring their rows of Q into shared memory
//   warp 16          MMA issuer, TMEM owner
//   warp 17          items, a record of each key tile (page scales), and its codes by TMA (a ring of
//                    two half tiles: K, V, K, ...)
//   warps 20-23      codes -> fp16 -> swizzled K and V tiles
// TMEM: S0 [0,128), S1 [128,256), O0 [256,256+DV), O1 [384,384+DV); W over the first half of each 64
// columns of S.
// Every wait is bounded; on a timeout the roles leave their loops and the CTA frees its TMEM.
#include <cuda_fp16.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "cache.h"
#include "common.cuh"

namespace bpa {
namespace {

constexpr int kThreads = 768;
constexpr int BN = 128;               // keys of a tile
constexpr int kRows = 256;            // rows of an item
constexpr int kMetas = 4;             // records of key tiles in flight
constexpr int kMma = 16, kAux = 17, kConv = 20;   // first warps of the roles
constexpr float kTau = 8.f, kOff = 7.f;
constexpr float kFar = 40.f;          // log2: a scale further from the item's first makes the request another kernel's
constexpr float kZeros = 20.f, kAllZeros = -kFar - kZeros;   // log2 scale of a page of zeros: below the largest so far; before any

struct TileMeta {
    int key0, len, end;
    uint32_t zero;                    // bit c: the v scale of chunk c is 0
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
    static constexpr int RBK = D < 128 ? D : 128, RBV = DV;      // bytes of a row of codes
    static constexpr int RAW = BN * (RBK > RBV ? RBK : RBV);     // half a tile of codes
    static constexpr int OFF_K = 2 * Q_BYTES, OFF_V = OFF_K + NS * K_BYTES, OFF_RAW = OFF_V + NS * V_BYTES;
    static constexpr int OFF_META = OFF_RAW + 2 * RAW, OFF_ITEM = OFF_META + kMetas * (int)sizeof(TileMeta);
    static constexpr int OFF_PAIR = OFF_ITEM + 2 * (int)sizeof(Item);           // flags of the softmax warps
    static constexpr int OFF_BAR = OFF_PAIR + 128;
    static constexpr int B_Q = 0, B_KF = 2, B_KE = B_KF + NS, B_VF = B_KE + NS, B_VE = B_VF + NS, B_S = B_VE + NS,
                         B_P = B_S + 2, B_O = B_P + 2, B_OE = B_O + 2, B_MF = B_OE + 2, B_ME = B_MF + kMetas,
                         B_IF = B_ME + kMetas, B_IE = B_IF + 2, B_RF = B_IE + 2, B_RE = B_RF + 2, B_PAIR = B_RE + 2,
                         B_FIN = B_PAIR + 8, NBAR = B_FIN + 1;
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

// Codes under a scale of 0: NaN stays NaN, whatever else they are counts as 0.
BPA_DEV uint32_t nan_or_0(uint32_t four) { return __vcmpeq4(four & 0x7f7f7f7fu, 0x7f7f7f7fu) & 0x7f7f7f7fu; }

// This thread's 64 scores of its row (columns c0 ..).  Rolled loops over 32 columns: the roles' code
// together has to stay in the instruction caches (unrolled, the warps spent two fifths of their time
// waiting for instructions).  EDGE: keys outside [kmin, kmax] are masked.

// The maxima of u and x.
template <bool EDGE>
BPA_DEV void maxima(uint32_t tS, const TileMeta* mt, int c0, float f_row, int k0, int kmin, int kmax, float& umax, float& xmax) {
    umax = xmax = -INFINITY;
#pragma unroll 1
    for (int c = c0; c < c0 + 64; c += 32) {
        uint32_t s[32];
        tmem_ld32(tS + c, s);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float a = f_row * mt->a[c / 16 + h];
            float mx = -INFINITY;
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
                float s0 = __uint_as_float(s[16 * h + i]), s1 = __uint_as_float(s[16 * h + i + 1]);
                if (EDGE) {
                    const int k = k0 + c + 16 * h + i;
                    s0 = k < kmin || k > kmax ? -INFINITY : s0 * a;
                    s1 = k + 1 < kmin || k + 1 > kmax ? -INFINITY : s1 * a;
                }
                mx = fmax3(mx, s0, s1);
            }
            const float x = EDGE ? mx : mx * a;                   // a >= 0
            umax = fmaxf(umax, x + mt->lv[c / 16 + h]);
            xmax = fmaxf(xmax, x);
        }
    }
}

// The weights as fp16 pairs over the scores (columns c0 .. c0 + 31); returns their sum of W e.
template <bool EDGE>
BPA_DEV float weights(uint32_t tS, const TileMeta* mt, int c0, float f_row, float mref, int k0, int kmin, int kmax) {
    float sum = 0.f;
#pragma unroll 1
    for (int cc = 0; cc < 2; ++cc) {
        const int c = c0 + 32 * cc;
        uint32_t s[32], pk[16];
        tmem_ld32(tS + c, s);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const float a = f_row * mt->a[c / 16 + h], b = mt->lv[c / 16 + h] - mref;
            const uint64_t a2 = f2_pack(a, a), b2 = f2_pack(b, b);
            uint64_t r2 = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                float y0, y1;
                f2_unpack(ffma2(f2_pack(__uint_as_float(s[16 * h + 2 * i]), __uint_as_float(s[16 * h + 2 * i + 1])), a2, b2), y0, y1);
                if (EDGE) {
                    const int k = k0 + c + 16 * h + 2 * i;
                    y0 = k < kmin || k > kmax ? -INFINITY : y0;
                    y1 = k + 1 < kmin || k + 1 > kmax ? -INFINITY : y1;
                }
                const float w0 = ex2(y0), w1 = ex2(y1);
                r2 = fadd2(r2, f2_pack(w0, w1));
                pk[8 * h + i] = h2(w0, w1);
            }
            float p, q;
            f2_unpack(r2, p, q);
            sum = fmaf(p + q, mt->e[c / 16 + h], sum);
        }
        tmem_st16_nowait(tS + c0 + 16 * cc, pk);
    }
    tmem_st_wait();
    return sum;
}

template <int D, int DV>
__global__ void __launch_bounds__(kThreads, 1) k_cache_attn_tc(const __grid_constant__ CUtensorMap tmK,
    const __grid_constant__ CUtensorMap tmV, const CacheAttnArgs a, uint32_t* counter, uint32_t* far, int vec_q, int vec_o) {
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
            mbar_init(BAR(C::B_Q + i), 256);
            mbar_init(BAR(C::B_S + i), 1);
            mbar_init(BAR(C::B_P + i), 256);
            mbar_init(BAR(C::B_O + i), 1);
            mbar_init(BAR(C::B_OE + i), 256);
            mbar_init(BAR(C::B_RF + i), 1);
            mbar_init(BAR(C::B_RE + i), 4);
            mbar_init(BAR(C::B_IF + i), 1);
            mbar_init(BAR(C::B_IE + i), 17);       // MMA warp, sixteen softmax warps
        }
        for (int i = 0; i < C::NS; ++i) {
            mbar_init(BAR(C::B_KF + i), 4);
            mbar_init(BAR(C::B_KE + i), 1);
            mbar_init(BAR(C::B_VF + i), 4);
            mbar_init(BAR(C::B_VE + i), 1);
        }
        for (int i = 0; i < kMetas; ++i) {
            mbar_init(BAR(C::B_MF + i), 1);
            mbar_init(BAR(C::B_ME + i), 20);       // four converting and sixteen softmax warps
        }
        for (int i = 0; i < 8; ++i) mbar_init(BAR(C::B_PAIR + i), 2);
        mbar_init(BAR(C::B_FIN), 1);
        *abort = 0;
        fence_mbar_init();
    }
    if (warp == kMma) {
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

    if (warp >= kConv) {
        // ------------------------------------------------------------ codes -> fp16 tiles
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        const int wq = warp - kConv;
        // half a tile from the ring to a K or V tile: rows of RB bytes, 16 bytes of a row at a time
        auto convert = [&](const uint8_t* raw, auto rb, uint8_t* tile, int left) {
            constexpr int RB = decltype(rb)::value, PER = RB / 16, ROWS = 32 / PER;   // lanes of a row, rows of a warp's read
            const int c = lane % PER, r = lane / PER, flip = c >> 2;                  // flip: the halves of a row on other banks
            uint8_t* slab = tile + (c >> 2) * C::SUB;
#pragma unroll 2
            for (int i = 0; i < 32 / ROWS; ++i) {
                const int row = 32 * wq + ROWS * i + r;
                uint4 x = *reinterpret_cast<const uint4*>(raw + row * RB + 16 * c);
                if (row >= left) x = make_uint4(0, 0, 0, 0);       // slots past the last token may hold anything
                const uint4 lo = make_uint4(cvt_lo(x.x), cvt_hi(x.x), cvt_lo(x.y), cvt_hi(x.y));
                const uint4 hi = make_uint4(cvt_lo(x.z), cvt_hi(x.z), cvt_lo(x.w), cvt_hi(x.w));
                *reinterpret_cast<uint4*>(slab + sw128_offset(row, (c & 3) * 2 + flip)) = flip ? hi : lo;
                *reinterpret_cast<uint4*>(slab + sw128_offset(row, (c & 3) * 2 + 1 - flip)) = flip ? lo : hi;
            }
            fence_proxy_async_smem();
            __syncwarp();
        };
        for (int t = 0;; ++t) {
            const int st = t % C::NS, use = t / C::NS, sl = t % kMetas;
            if (!wait(C::B_MF + sl, t / kMetas, 0xE0) || metas[sl].end) break;
            const int left = metas[sl].len - metas[sl].key0;
            const uint32_t zero = metas[sl].zero >> (2 * wq) & 3;   // this warp's two 16 rows
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(C::B_ME + sl));
            if (!wait(C::B_RF, t, 0xE1) || (use > 0 && !wait(C::B_KE + st, use - 1, 0xE2))) break;
            convert(smem + C::OFF_RAW, std::integral_constant<int, C::RBK>(), smem + C::OFF_K + st * C::K_BYTES, left);
            if (lane == 0) {
                mbar_arrive(BAR(C::B_KF + st));
                mbar_arrive(BAR(C::B_RE));
            }
            if (!wait(C::B_RF + 1, t, 0xE3) || (use > 0 && !wait(C::B_VE + st, use - 1, 0xE4))) break;
            if (zero) {                // rare, and 5 % of the prompts' time inside the conversion's loop
#pragma unroll 1
                for (int i = lane; i < 2 * C::RBV; i += 32)       // a row is RBV / 16 pieces: 32 rows of them
                    if (zero >> (i / C::RBV) & 1) {
                        uint4* at = reinterpret_cast<uint4*>(smem + C::OFF_RAW + C::RAW + 32 * wq * C::RBV) + i;
                        *at = make_uint4(nan_or_0(at->x), nan_or_0(at->y), nan_or_0(at->z), nan_or_0(at->w));
                    }
                __syncwarp();
            }
            convert(smem + C::OFF_RAW + C::RAW, std::integral_constant<int, C::RBV>(), smem + C::OFF_V + st * C::V_BYTES, left);
            if (lane == 0) {
                mbar_arrive(BAR(C::B_VF + st));
                mbar_arrive(BAR(C::B_RE + 1));
            }
        }
    } else if (warp >= kMma) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp == kAux) {
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
                auto there = [&](int j) { return lane < 8 && j < tiles && (first + j) * BN + 16 * lane < rq.len; };
                auto page_of = [&](int j) { return there(j) ? table[((first + j) * BN + 16 * lane) / a.P] : -1; };
                auto scales_of = [&](int j, int& id, float& ks, float& vs) {
                    ks = vs = 0.f;
                    if (id >= 0 && id < a.num_pages) {
                        ks = a.kscale[static_cast<int64_t>(id) * a.Hkv + hk];
                        vs = a.vscale[static_cast<int64_t>(id) * a.Hkv + hk];
                    } else {
                        if (there(j)) report(a.status, ST_CHECK, 0xCE0);
                        id = -1;
                    }
                };
                int id = page_of(0), id1 = page_of(1);
                float ks, vs;
                scales_of(0, id, ks, vs);
                const unsigned some = __ballot_sync(0xffffffffu, vs > 0.f);
                const float lv0 = some ? __log2f(__shfl_sync(0xffffffffu, vs, __ffs(some) - 1)) : 0.f;
                if (lane == 0) {
                    *it = {1, rq.row0, rq.n, rq.len, hk, i0, first, tiles, lv0, {}};
                    mbar_arrive(BAR(C::B_IF + (k & 1)));
                }
                bool ok = true;
                float lvmax = -INFINITY;
                for (int j = 0; j < tiles; ++j, ++t) {
                    const int sl = t % kMetas, id2 = page_of(j + 2);
                    float ks1, vs1;
                    scales_of(j + 1, id1, ks1, vs1);
                    if (t >= kMetas && !(ok = wait(C::B_ME + sl, t / kMetas - 1, 0xE6))) break;
                    TileMeta* m = metas + sl;
                    const uint32_t zero = __ballot_sync(0xffffffffu, !(vs > 0.f));
                    float lv = vs > 0.f ? __log2f(vs) : -INFINITY;
                    if (vs > 0.f && !(fabsf(lv - lv0) <= kFar)) {
                        far[r] = 1;
                        lv = lv0;
                    }
                    lvmax = fmaxf(lvmax, lv);
#pragma unroll
                    for (int o = 1; o < 8; o <<= 1) lvmax = fmaxf(lvmax, __shfl_xor_sync(0xffffffffu, lvmax, o));
                    if (lv == -INFINITY) lv = lvmax == -INFINITY ? kAllZeros : lvmax - kZeros;
                    if (lane < 8) {
                        m->a[lane] = ks * a.scale * kLog2e;
                        m->lv[lane] = lv;
                        m->e[lane] = ex2(lv0 - lv);
                    }
                    if (lane == 0) {
                        m->key0 = (first + j) * BN;
                        m->len = rq.len;
                        m->end = 0;
                        m->zero = zero;
                    }
                    __syncwarp();
                    if (lane == 0) mbar_arrive(BAR(C::B_MF + sl));
                    // the tile's codes: K, then V, 16 keys a copy
                    const int n = __popc(__ballot_sync(0xffffffffu, id >= 0));
                    const int tok = ((first + j) * BN + 16 * lane) % a.P;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const int rb = kv ? C::RBV : C::RBK;
                        if (t > 0 && !(ok = wait(C::B_RE + kv, t - 1, 0xEF))) break;
                        if (lane == 0) mbar_expect_tx(BAR(C::B_RF + kv), n * 16 * rb);
                        __syncwarp();
                        if (id >= 0)
                            tma_load_4d(sb + C::OFF_RAW + kv * C::RAW + 16 * lane * rb, kv ? &tmV : &tmK, BAR(C::B_RF + kv), 0, tok, hk, id);
                    }
                    if (!ok) break;
                    id = id1;
                    ks = ks1;
                    vs = vs1;
                    id1 = id2;
                }
                if (!ok) break;
            }
            if (t > 0 && *abort) {     // after a timeout: the copies in flight end before the CTA does
                int never = 0;
                for (int kv = 0; kv < 2; ++kv)
                    for (int p = t - 1; p <= t; ++p) mbar_wait(BAR(C::B_RF + kv), p & 1, &never, a.status, 0xEF);
            }
            publish_end();
        } else if (warp == kMma) {
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
#pragma unroll 4
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * C::SUB + (kk & 3) * 32;
                        tc_mma_ss_w(tmem + i * BN, sdesc_advance(qd, off), sdesc_advance(kd, off), C::IDESC_S, kk > 0);
                    }
                    tc_commit_w(BAR(C::B_S + i));
                };
                auto issue_pv = [&](int i, int pos, bool first) {
                    const uint64_t vd = sdesc_sw128(sb + C::OFF_V + pos % C::NS * C::V_BYTES, C::SUB, 1024);
#pragma unroll 4
                    for (int kk = 0; kk < BN / 16; ++kk)       // the weights of 64 keys lie over the first half of their scores
                        tc_mma_ts_w(tmem + 256 + i * 128, tmem + i * BN + kk * 8 + (kk >> 2) * 32, sdesc_advance(vd, kk * 2048), C::IDESC_PV,
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
        // ------------------------------------------------------------ softmax: two threads own a row, 64 columns each
        asm volatile("setmaxnreg.inc.sync.aligned.u32 88;");
        const int qt = warp >> 3, half = (warp >> 2) & 1, row = (warp & 3) * 32 + lane, c0 = 64 * half;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t tS = tmem + qt * BN + lanes, tO = tmem + 256 + qt * 128 + lanes;
        // the two warps of 32 rows meet at a barrier of their own and tell each other whether a row moves its M
        const int pair = qt * 4 + (warp & 3);
        volatile int* flags = reinterpret_cast<volatile int*>(smem + C::OFF_PAIR) + 4 * pair;
        int meets = 0;
        auto meet = [&]() {
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(C::B_PAIR + pair));
            return wait(C::B_PAIR + pair, meets++, 0xF4);
        };
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
            int kmin = 0, kmax = INT_MAX;      // a row that is not there masks nothing (q = 0)
            if (there) row_keys(a, Req{it.row0, it.n, it.len, false}, tok, kmin, kmax);
            float f_row = 1.f;
            if (busy && it.tiles) {
                // ---- the row of q as fp16, its largest value scaled into [2^7, 2^8): all of it for the
                // largest, this thread's half to store
                const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + static_cast<int64_t>(it.row0 + tok) * a.qs[0] +
                                         static_cast<int64_t>(head) * a.qs[1];
                auto piece = [&](int c) {
                    uint4 x = make_uint4(0, 0, 0, 0);
                    if (there && 8 * c < a.d) {
                        if (vec_q) {
                            x = *reinterpret_cast<const uint4*>(q + 8 * c);
                        } else {
                            uint32_t w[4];
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                const unsigned short* p = reinterpret_cast<const unsigned short*>(q + 8 * c + 2 * e);
                                w[e] = p[0] | static_cast<uint32_t>(p[1]) << 16;
                            }
                            x = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                    return x;
                };
                uint32_t top = 0;
                auto largest = [&](const uint4& x) {
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fff0000u, (w[e] << 16) & 0x7fff0000u));
                };
                uint4 x[D / 16];
#pragma unroll
                for (int c = 0; c < D / 16; ++c) x[c] = piece(half * (D / 16) + c);
#pragma unroll 4
                for (int c = 0; c < D / 16; ++c) largest(piece((1 - half) * (D / 16) + c));
#pragma unroll
                for (int c = 0; c < D / 16; ++c) largest(x[c]);
                int ex = top && top < 0x7f800000u ? static_cast<int>(top >> 23) - 127 - 7 : 0;
                ex = min(max(ex, -126), 126);
                const float up = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
                f_row = __uint_as_float(static_cast<uint32_t>(127 + ex) << 23);
                uint8_t* tile = smem + qt * C::Q_BYTES;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    const int c = half * (D / 16) + i;
                    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
                    uint32_t y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        y[e] = h2(__uint_as_float(w[e] << 16) * up, __uint_as_float(w[e] & 0xffff0000u) * up);
                    *reinterpret_cast<uint4*>(tile + (c >> 3) * C::SUB + sw128_offset(row, c & 7)) = make_uint4(y[0], y[1], y[2], y[3]);
                }
                fence_proxy_async_smem();
                mbar_arrive(BAR(C::B_Q + qt));
            }
            float M = -INFINITY, xm = -INFINITY, L = 0.f;      // M of the row; x and L of this thread's columns
            for (int j = 0; j < it.tiles; ++j, ++t) {
                const int sl = t % kMetas, k0 = (it.first + j) * BN;
                if (!(ok = wait(C::B_MF + sl, t / kMetas, 0xF1))) break;
                if (!busy) {                   // no rows: only the record's turn
                    if (lane == 0) mbar_arrive(BAR(C::B_ME + sl));
                    continue;
                }
                if (!(ok = wait(C::B_S + qt, cs, 0xF2))) break;
                ++cs;
                tc_fence_after();
                const TileMeta* mt = metas + sl;
                const bool edge = __any_sync(0xffffffffu, k0 < kmin || k0 + BN - 1 > kmax);
                float um, x;
                if (edge) maxima<true>(tS, mt, c0, f_row, k0, kmin, kmax, um, x);
                else maxima<false>(tS, mt, c0, f_row, k0, kmin, kmax, um, x);
                xm = fmaxf(xm, x);
                bool move = j == 0;
                if (!move) {                   // does a row of the two warps move its M?
                    volatile int* f = flags + 2 * (t & 1);
                    const int mine = __any_sync(0xffffffffu, um > M + kTau);
                    if (lane == 0) f[half] = mine;
                    if (!(ok = meet())) break;
                    move = f[0] | f[1];
                }
                if (move) {                    // both threads of a row take the maximum of u over all of its columns
                    float u2, x2;
                    if (edge) maxima<true>(tS, mt, 64 - c0, f_row, k0, kmin, kmax, u2, x2);
                    else maxima<false>(tS, mt, 64 - c0, f_row, k0, kmin, kmax, u2, x2);
                    um = fmaxf(um, u2);
                    float fac = 1.f;
                    if (um > M + kTau) {
                        fac = M == -INFINITY ? 0.f : ex2(M - um);
                        M = um;
                        L *= fac;
                    }
                    if (j > 0) {               // S(j) is complete, so every earlier W V has been added to O
#pragma unroll 1
                        for (int cc = half * (DV / 64); cc < (half + 1) * (DV / 64); ++cc) {
                            uint32_t r[32];
                            tmem_ld32(tO + cc * 32, r);
#pragma unroll
                            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * fac);
                            tmem_st32(tO + cc * 32, r);
                        }
                    }
                    if (!(ok = meet())) break; // the other thread has read this one's scores
                }
                const float mref = M == -INFINITY ? 0.f : M - kOff;
                L += edge ? weights<true>(tS, mt, c0, f_row, mref, k0, kmin, kmax) : weights<false>(tS, mt, c0, f_row, mref, k0, kmin, kmax);
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
                // the other half of the row, by way of the tile of Q, which every product has read
                float2* rows2 = reinterpret_cast<float2*>(smem + qt * C::Q_BYTES);
                rows2[128 * half + row] = make_float2(L, xm);
                if (!(ok = meet())) break;
                const float2 other = rows2[128 * (1 - half) + row];
                // the same sum on both threads
                L = L + other.x;
                xm = fmaxf(xm, other.y);
                if (!(ok = meet())) break;
            }
            // ---- epilogue: o = O 2^lv0 / L; l relative to the row's maximum of x
            float l = M == -INFINITY ? (L != L ? L : 0.f) : L * ex2(M - kOff - it.lv0 - xm), mm = xm, part = 1.f;
            if (a.sink) {
                const float sk = __ldg(a.sink + head) * kLog2e, nm = fmaxf(xm, sk);
                const float old = l;
                l = (xm == -INFINITY ? l : l * ex2(xm - nm)) + ex2(sk - (nm == -INFINITY ? 0.f : nm));
                part = xm == -INFINITY || old == 0.f ? (old != old ? old : 0.f) : old * ex2(xm - nm) / l;   // what the keys have of the row
                mm = nm;
            }
            // two factors: 2^lv0 / L alone may be below float32's normal numbers
            const float inv = (L == 0.f || M == -INFINITY ? (L != L ? L : 0.f) : 1.f / L) * part, s0 = ex2(it.lv0);
            const int64_t out_row = it.row0 + tok;
            if (there && a.m && half == 0) {
                a.m[static_cast<int64_t>(head) * a.T + out_row] = mm == -INFINITY ? mm : mm * kLn2;
                a.l[static_cast<int64_t>(head) * a.T + out_row] = l;
            }
            __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o) + out_row * a.os[0] + static_cast<int64_t>(head) * a.os[1];
#pragma unroll 1
            for (int cc = half * (DV / 64); cc < (half + 1) * (DV / 64); ++cc) {
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
                    for (int e = 0; e < 4; ++e) w[e] = pack_bf16(__uint_as_float(r[8 * v + 2 * e]) * inv * s0, __uint_as_float(r[8 * v + 2 * e + 1]) * inv * s0);
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
    if (warp == kMma) {
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, int DV>
cudaError_t launch(const CacheAttnArgs& a, const CUtensorMap* maps, uint32_t* counter, uint32_t* far, cudaStream_t s) {
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
    k_cache_attn_tc<D, DV><<<static_cast<unsigned>(std::min<int64_t>(n, most)), kThreads, C::SMEM, s>>>(maps[0], maps[1], a, counter,
                                                                                                       far, vec_q, vec_o);
    return cudaGetLastError();
}

}  // namespace

bool cache_attn_tc_takes(const CacheAttnArgs& a) {
    if (a.dtype != BPA_BF16 || a.d % 16 || a.dv % 16 || a.d > 128 || a.dv > 128 || (a.d <= 64 && a.dv > 64) || a.P % 16) return false;
    const int64_t rows = static_cast<int64_t>(a.max_q) * a.G;
    if (rows <= kFewRows) return false;
    // An item's keys are not shared between CTAs here, as they are in the kernel for few rows: with few
    // items (one token of 128 heads over a long context) that one fills the GPU and this one does not.
    // With all CTAs busy this one is 4.6 times faster (pieces of prompts 1,540 us and 7.1 ms).  The border, one
    // request over 131,072 tokens, 4 q heads on each of 8 kv heads, this kernel and that one: 16 items
    // (128 tokens) 2,383 and 1,367 us, 24 items 2,387 and 2,036, 32 items 2,388 and 2,703; over 4,096 tokens 16
    // items 108 and 70 us, 32 items 109 and 118; four requests over 8,192, 32 items 184 and 199 us, but 155 and
    // 113 where the items are half full (32 tokens).
    const int64_t items = std::min(a.R * ((rows + kRows - 1) / kRows), static_cast<int64_t>(a.T) * a.G / kRows + a.R) * a.Hkv;
    return items >= 32;
}

CacheBox cache_attn_tc_box(const CacheAttnArgs& a) { return {a.d <= 64 ? 64 : 128, a.dv <= 64 ? 64 : 128, 16}; }

cudaError_t launch_cache_attn_tc(const CacheAttnArgs& a, const CUtensorMap* maps, uint32_t* counter, uint32_t* far, cudaStream_t s) {
    if (a.d <= 64) return launch<64, 64>(a, maps, counter, far, s);
    return a.dv <= 64 ? launch<128, 64>(a, maps, counter, far, s) : launch<128, 128>(a, maps, counter, far, s);
}

}  // namespace bpa
