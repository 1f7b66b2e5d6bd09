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
// Bounded by the chain from scores to weights and back through the products (compute, not bytes): about
// three instructions and one exponential a score, and the products' operands and the conversion share the
// shared memory's ports.  Two threads share a row (64 columns each), so sixteen warps work on the softmax and
// cover each other's latencies.  Its loops stay rolled, code that runs once an item too, and what waits seldom
// do is a function of its own: the roles' code has to stay in the instruction caches (straight code for an item's
// rows of q waited 9 us for its instructions).  One thread issues all products (eight of them took a whole warp
// that elects a lane for each 800 cycles, 1,539 us for the prompts below).  Five pieces of prompts, 6,852 rows of 32
// heads over up to 16,000 tokens, 128 channels: 1,339 us, 1,055 TFLOP/s (the kernel for few rows 7,225).
//
// Trees of drafted tokens (TREE): the keys of the step are seen by mask, and as a step has few rows and long contexts, items
// are cut between CTAs by cost; their pieces go to the workspace for the join of cache_attn_mma.cuh.  32 requests of 8 to 64
// rows, 4 q heads on each of 8 kv heads, 200 to 8,191 tokens: 199 us in all (555 TFLOP/s; the kernel for few rows 720); two
// of 40 and 64 rows over 100,000 and more 277 us, 817 TFLOP/s (1,486).
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
#include "cache_attn_mma.cuh"
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
    int slot, alt, pad;               // trees: place of a piece (-1: a whole item), even and odd key tiles apart
};
using cache_mma::kMaxTcCtas;
using cache_mma::Pieces;
using cache_mma::Rec;

// mbar_wait with what is done seldom in a function of its own: the roles' loops have to stay in the instruction caches.
// 0: give up.
__device__ __noinline__ uint64_t give_up(uint64_t t0, volatile int* abort, uint32_t* status, uint32_t where) {
    const uint64_t now = globaltimer();
    if (*abort) return 0;
    if (t0 == 1) return now;
    if (now - t0 <= kWaitLimitNs) return t0;
    *abort = 1;
    report(status, ST_TIMEOUT, where);
    return 0;
}
BPA_DEV bool bounded_wait(uint32_t bar, uint32_t parity, volatile int* abort, uint32_t* status, uint32_t where) {
    uint64_t t0 = 1;
    for (uint32_t it = 1; !mbar_try_wait(bar, parity); ++it)
        if ((it & 63u) == 0 && (t0 = give_up(t0, abort, status, where)) == 0) return false;
    return true;
}

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
    static constexpr int OFF_EXP = OFF_PAIR + 128;               // exponents of the rows of q, 8 x 32
    static constexpr int OFF_BAR = OFF_EXP + 256;
    static constexpr int B_Q = 0, B_KF = 2, B_KE = B_KF + NS, B_VF = B_KE + NS, B_VE = B_VF + NS, B_S = B_VE + NS,
                         B_P = B_S + 2, B_O = B_P + 2, B_OE = B_O + 2, B_MF = B_OE + 2, B_ME = B_MF + kMetas,
                         B_IF = B_ME + kMetas, B_IE = B_IF + 2, B_RF = B_IE + 2, B_RE = B_RF + 2, B_PAIR = B_RE + 2,
                         B_FIN = B_PAIR + 8, B_X = B_FIN + 1, NBAR = B_X + 1;
    static constexpr int SMEM = 1024 + OFF_BAR + 8 * NBAR + 16;
    static_assert(SMEM <= 232448, "shared memory");
    static constexpr uint32_t F16 = 1u << 4;                     // float32 sums, both operands fp16
    static constexpr uint32_t IDESC_S = F16 | (BN >> 3) << 17 | (128 >> 4) << 24;
    static constexpr uint32_t IDESC_PV = F16 | 1u << 16 | (DV >> 3) << 17 | (128 >> 4) << 24;   // V: MN-major
};

// Keys of one copy: whatever of a tile one page is sure to hold.
__host__ __device__ inline int box_rows(int P) { return P % 128 == 0 ? 128 : P % 64 == 0 ? 64 : P % 32 == 0 ? 32 : 16; }

// A request's items: nothing for one that the kernel for few rows takes.
BPA_DEV int groups_of(const CacheAttnArgs& a, const Req& q) {
    const int rows = q.n * a.G;
    return rows > (a.tree ? kFewTreeRows : kFewRows) ? (rows + kRows - 1) / kRows : 0;
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
// waiting for instructions).  EDGE 1: keys outside [kmin, kmax] are masked; 2 (trees): those whose bit of `seen` is not set.
enum { E_NONE = 0, E_RANGE = 1, E_BITS = 2 };
template <int EDGE>
BPA_DEV bool masked(int k, int kmin, int kmax, uint32_t seen, int bit) {
    return EDGE == E_RANGE ? k < kmin || k > kmax : !(seen >> bit & 1);
}

// The maxima of u and x.
template <int EDGE>
BPA_DEV void maxima(uint32_t tS, const TileMeta* mt, int c0, float f_row, int k0, int kmin, int kmax, uint64_t seen, float& umax, float& xmax) {
    umax = xmax = -INFINITY;
#pragma unroll 1
    for (int c = c0; c < c0 + 64; c += 32) {
        uint32_t s[32];
        const uint32_t bits = static_cast<uint32_t>(seen >> (c - c0));
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
                    s0 = masked<EDGE>(k, kmin, kmax, bits, 16 * h + i) ? -INFINITY : s0 * a;
                    s1 = masked<EDGE>(k + 1, kmin, kmax, bits, 16 * h + i + 1) ? -INFINITY : s1 * a;
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
template <int EDGE>
BPA_DEV float weights(uint32_t tS, const TileMeta* mt, int c0, float f_row, float mref, int k0, int kmin, int kmax, uint64_t seen) {
    float sum = 0.f;
#pragma unroll 1
    for (int cc = 0; cc < 2; ++cc) {
        const int c = c0 + 32 * cc;
        const uint32_t bits = static_cast<uint32_t>(seen >> (32 * cc));
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
                    y0 = masked<EDGE>(k, kmin, kmax, bits, 16 * h + 2 * i) ? -INFINITY : y0;
                    y1 = masked<EDGE>(k + 1, kmin, kmax, bits, 16 * h + 2 * i + 1) ? -INFINITY : y1;
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

// Trees: which of the 64 keys from k0 on the row sees.
BPA_DEV uint64_t seen_from(const TreeRow& t, int k0, int len) {
    auto ones = [](int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; };
    auto word = [&](int w) { return w < t.words ? __ldg(t.bits + w) : 0u; };
    if (k0 >= len) return 0;
    uint64_t seen = ones(t.ctx - k0) & ~ones(t.lo - k0);      // in front of the step's tokens
    const int j = k0 - t.ctx;                                 // of the step's tokens, the first here
    if (j >= 0) {
        const int w = j >> 5;
        const uint32_t a = word(w), b = word(w + 1), c = word(w + 2);
        seen = __funnelshift_r(a, b, j & 31) | static_cast<uint64_t>(__funnelshift_r(b, c, j & 31)) << 32;
    } else if (j > -64) {
        seen |= (word(0) | static_cast<uint64_t>(word(1)) << 32) << -j;
    }
    return seen & ones(len - k0);
}

// Trees: items are cut between CTAs.  Each takes an equal share of the cost of all items (a key tile counts what its
// rows take, an item's start and end kExtra), as in the kernel for few rows, and leaves pieces of items
// for the same join.  An item of up to 128 rows has its even key tiles on one row tile and its odd ones on the other, the same rows on
// both, so that all warps work; they are added up at its end.  Measured: a tile of 256 rows 2.3 us, one of 128 1.75, an item's
// start and end about 10 (kExtra 4, 8, 14 and 20: 32 requests of 64 rows over 200 to 8,191 tokens 248, 240, 218 and 205 us,
// those of 8 to 64 rows 214, 203, 193 and 194).
constexpr int kTwo = 4, kAlt = 3, kExtra = 18;
struct Cut {                          // of an item: first key tile, tiles (at least one), what a tile counts for
    int first, n, each;
    bool keys;                        // no: the one tile is none
    BPA_DEV int cost() const { return n * each + kExtra; }
    BPA_DEV int within(long long c) const { return c <= kExtra ? 0 : (static_cast<int>(c) - kExtra) / each; }
};
BPA_DEV Cut cut_of(const CacheAttnArgs& a, const Req& q, int g) {
    int lo, hi;
    tree_span(a, q, lo, hi);
    const int each = q.n * a.G - g * kRows > 128 ? kTwo : kAlt;
    if (lo > hi) return {0, 1, each, false};
    return {lo / BN, hi / BN - lo / BN + 1, each, true};
}
BPA_DEV long long cost_of(const CacheAttnArgs& a, const Req& q) {
    const int groups = groups_of(a, q);
    if (groups == 0) return 0;
    return ((groups - 1) * static_cast<long long>(cut_of(a, q, 0).cost()) + cut_of(a, q, groups - 1).cost()) * a.Hkv;
}

// TREE: of the kernel's CTAs, what the join of their pieces reads; otherwise empty.
template <int D, int DV, bool TREE>
__global__ void __launch_bounds__(kThreads, 1) k_cache_attn_tc(const __grid_constant__ CUtensorMap tmK,
    const __grid_constant__ CUtensorMap tmV, const CacheAttnArgs a, uint32_t* counter, uint32_t* far, int vec_q, int vec_o,
    const Pieces pieces) {
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
        mbar_init(BAR(C::B_X), 16);            // the softmax warps
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
        return __all_sync(0xffffffffu, bounded_wait(BAR(b), parity & 1, abort, a.status, where)) != 0;
    };

    if (warp >= kConv) {
        // ------------------------------------------------------------ codes -> fp16 tiles
        asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        const int wq = warp - kConv;
        // Half a tile from the ring to a K or V tile: rows of RB bytes, 16 bytes of a row at a time, four reads under way
        // together.  Eight lanes in a row take two rows (RB 128: the halves of them that lie on other banks),
        // whose swizzled units lie on other banks too, so that neither side has conflicts, and every address is a
        // base and a constant.
        auto convert = [&](const uint8_t* raw, auto rb, uint8_t* tile, int left) {
            constexpr int RB = decltype(rb)::value, STEP = RB == 128 ? 4 : 8;         // rows of a warp's read
            const int c = lane & 3, p = lane >> 2 & 1, q = lane >> 4;
            const int slab = RB == 128 ? (lane >> 3 & 1) ^ p : 0, r = RB == 128 ? 2 * q + p : lane >> 2;
            const uint8_t* from = raw + (32 * wq + r) * RB + 64 * slab + 16 * c;
            uint8_t* to = tile + slab * C::SUB + (32 * wq + r) * 128;
            const int o = (2 * c ^ r) << 4;                                           // unit 2 c of the row; 2 c + 1: o ^ 16
            uint8_t* const at[4] = {to + o, to + (o ^ 16), to + (o ^ 64), to + (o ^ 80)};
            const int rows = left - 32 * wq - r;                                      // slots past the last token may hold anything
            auto four = [&](int i0, auto tail) {
                uint4 x[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const uint4*>(from + (i0 + i) * STEP * RB);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (decltype(tail)::value && (i0 + i) * STEP >= rows) x[i] = make_uint4(0, 0, 0, 0);
                    // rows four further on are swizzled the other way
                    const int flip = RB == 128 ? 2 * (i & 1) : 0;
                    *reinterpret_cast<uint4*>(at[flip] + (i0 + i) * STEP * 128) =
                        make_uint4(cvt_lo(x[i].x), cvt_hi(x[i].x), cvt_lo(x[i].y), cvt_hi(x[i].y));
                    *reinterpret_cast<uint4*>(at[flip + 1] + (i0 + i) * STEP * 128) =
                        make_uint4(cvt_lo(x[i].z), cvt_hi(x[i].z), cvt_lo(x[i].w), cvt_hi(x[i].w));
                }
            };
#pragma unroll 1
            for (int i0 = 0; i0 < 32 / STEP; i0 += 4) {
                if (32 * wq + 32 > left) four(i0, std::true_type());
                else four(i0, std::false_type());
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
            const int box = box_rows(a.P);
            int t = 0;                 // records written
            auto publish_end = [&]() {
                if (t >= kMetas && !wait(C::B_ME + t % kMetas, t / kMetas - 1, 0xE4)) return;
                if (lane == 0) {
                    metas[t % kMetas].end = 1;
                    mbar_arrive(BAR(C::B_MF + t % kMetas));
                }
            };
            // trees: this CTA's share of the cost of all items, and its pieces one after the other
            struct {
                int r, hk, g, groups;
                Req rq;
                long long total, at, off, left;
                int parts;
                bool first;
                Rec rec;
            } own = {};
            if (TREE) {
                long long total = 0;
                for (int r = lane; r < a.R; r += 32) total += cost_of(a, request_of(a, r));
#pragma unroll
                for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
                const int ctas = gridDim.x, cta = blockIdx.x;
                // a share is at least a tile among the CTAs that take part, so the pieces of an item lie side by side
                own.parts = static_cast<int>(min(total / kTwo, static_cast<long long>(ctas)));
                own.total = total;
                const long long begin = cta < own.parts ? cache_mma::share(total, cta, own.parts) : total;
                own.left = (cta < own.parts ? cache_mma::share(total, cta + 1, own.parts) : total) - begin;
                own.at = begin;
                own.first = true;
                long long before = 0;
                for (int base = 0; own.left > 0 && base < a.R; base += 32) {
                    const long long c = base + lane < a.R ? cost_of(a, request_of(a, base + lane)) : 0;
                    long long x = c;
#pragma unroll
                    for (int o = 1; o < 32; o <<= 1) {
                        const long long y = __shfl_up_sync(0xffffffffu, x, o);
                        if (lane >= o) x += y;
                    }
                    const unsigned hit = __ballot_sync(0xffffffffu, begin < before + x);
                    if (hit) {
                        const int src = __ffs(hit) - 1;
                        own.r = base + src;
                        own.off = begin - before - __shfl_sync(0xffffffffu, x - c, src);
                        break;
                    }
                    before += __shfl_sync(0xffffffffu, x, 31);
                }
                if (own.left > 0) {
                    own.rq = request_of(a, own.r);
                    own.groups = groups_of(a, own.rq);
                    const long long per_head = cost_of(a, own.rq) / a.Hkv;
                    own.hk = static_cast<int>(own.off / per_head);
                    own.off -= own.hk * per_head;
                    while (own.g + 1 < own.groups && own.off >= cut_of(a, own.rq, own.g).cost()) own.off -= cut_of(a, own.rq, own.g++).cost();
                }
            }
            // the next piece: key tiles [t0, t1) of item (own.r, own.hk, g)
            auto next_piece = [&](int& g, int& t0, int& t1, int& slot, Cut& cut) {
                while (own.left > 0) {
                    if (!own.first && ++own.g == own.groups) {
                        own.g = 0;
                        if (++own.hk == a.Hkv) {
                            own.hk = 0;
                            do {
                                if (++own.r >= a.R) {      // only if the lengths changed during the call
                                    if (lane == 0) report(a.status, ST_CHECK, 0xCE5);
                                    own.left = 0;
                                    return false;
                                }
                                own.rq = request_of(a, own.r);
                                own.groups = groups_of(a, own.rq);
                            } while (own.groups == 0);
                        }
                    }
                    own.first = false;
                    cut = cut_of(a, own.rq, own.g);
                    const long long off = own.off, to = min(static_cast<long long>(cut.cost()), off + own.left);
                    g = own.g;
                    t0 = cut.within(off);
                    t1 = cut.within(to);
                    const bool lead = t0 > 0, trail = t1 < cut.n;
                    slot = lead ? 2 * static_cast<int>(blockIdx.x) : trail ? 2 * static_cast<int>(blockIdx.x) + 1 : -1;
                    if (t0 < t1 && trail && !lead) {
                        // its pieces: up to the last CTA c with total c / parts < the end of the item's cost
                        const long long at_end = own.at + (cut.cost() - off);
                        own.rec.trail = static_cast<int>((at_end * own.parts + own.total - 1) / own.total) - blockIdx.x;
                        own.rec.r = own.r;
                        own.rec.row0 = own.rq.row0;
                        own.rec.hk = own.hk;
                        own.rec.i0 = g * kRows;
                        own.rec.nrows = min(own.rq.n * a.G - g * kRows, kRows);
                    }
                    own.left -= to - off;
                    own.at += to - off;
                    own.off = 0;
                    if (t0 < t1) return true;
                }
                return false;
            };
            for (int k = 0;; ++k) {
                if (k >= 2 && !wait(C::B_IE + (k & 1), (k >> 1) - 1, 0xE5)) break;
                Req rq = {};
                int r = -1, groups = 0;
                uint32_t idx = 0;
                int g = 0, t0 = 0, t1 = 0, slot = -1;
                Cut cut = {};
                if (TREE) {
                    if (next_piece(g, t0, t1, slot, cut)) {
                        r = own.r;
                        rq = own.rq;
                    }
                } else {
                if (lane == 0) idx = atomicAdd(counter, 1u);
                idx = __shfl_sync(0xffffffffu, idx, 0);
                // the item's request: a running sum over the requests, 32 at a time
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
                const int hk = TREE ? own.hk : idx % a.Hkv;
                const int i0 = (TREE ? g : groups - 1 - static_cast<int>(idx / a.Hkv)) * kRows;   // last rows first
                int first, tiles;
                if (TREE) {
                    first = cut.first + t0;
                    tiles = cut.keys ? t1 - t0 : 0;
                } else {
                    const int last = min(rq.n * a.G, i0 + kRows) - 1;
                    int lo, hi, y;
                    row_keys(a, rq, i0 / a.G, lo, y);
                    row_keys(a, rq, last / a.G, y, hi);
                    first = lo <= hi ? lo / BN : 0;
                    tiles = lo <= hi ? hi / BN - first + 1 : 0;
                }
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
                    *it = {1, rq.row0, rq.n, rq.len, hk, i0, first, tiles, lv0, slot, TREE && rq.n * a.G - i0 <= 128, 0};
                    mbar_arrive(BAR(C::B_IF + (k & 1)));
                }
                if (TREE) {            // the item's rows of q on their way to L2: the softmax warps come to them a tile or more later
                    const int rows = min(rq.n * a.G - i0, kRows), lines = (a.d * 2 + 127) / 128;
                    for (int i = lane; i < rows * lines; i += 32) {
                        const int ri = i0 + i / lines, tok = ri / a.G;
                        const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + static_cast<int64_t>(rq.row0 + tok) * a.qs[0] +
                                                 static_cast<int64_t>(hk * a.G + ri - tok * a.G) * a.qs[1];
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const uint8_t*>(q) + 128 * (i % lines)));
                    }
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
                    if (zero & 0xffu) {
#pragma unroll
                        for (int o = 1; o < 8; o <<= 1) lvmax = fmaxf(lvmax, __shfl_xor_sync(0xffffffffu, lvmax, o));
                    }
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
                    // the tile's codes: K, then V, a box of keys (of one page) a copy
                    const int tok = ((first + j) * BN + 16 * lane) % a.P;
                    const bool copies = id >= 0 && 16 * lane % box == 0;
                    const int n = __popc(__ballot_sync(0xffffffffu, copies)) * box;
#pragma unroll
                    for (int kv = 0; kv < 2; ++kv) {
                        const int rb = kv ? C::RBV : C::RBK;
                        if (t > 0 && !(ok = wait(C::B_RE + kv, t - 1, 0xEF))) break;
                        if (lane == 0) mbar_expect_tx(BAR(C::B_RF + kv), n * rb);
                        __syncwarp();
                        if (copies)
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
            if (TREE && lane == 0) pieces.recs[blockIdx.x] = own.rec;
        } else if (warp == kMma) {
            // -------------------------------------------------------- MMA issuer
            // One thread (the elected one) waits, issues and commits: with the whole warp in step and a lane elected for
            // each product, eight of them took 800 cycles.
            uint32_t leader;
            asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\tselp.u32 %0, 1, 0, e;\n\t}" : "=r"(leader));
            if (leader) {
            auto wait = [&](int b, int parity, uint32_t where) { return bounded_wait(BAR(b), parity & 1, abort, a.status, where); };
            int t = 0, np[2] = {0, 0}, seen[2] = {0, 0};   // key tiles; W tiles used, items with work, per row tile
            bool ok = true;
            for (int k = 0; ok; ++k) {
                if (!wait(C::B_IF + (k & 1), k >> 1, 0xE7)) break;
                const Item it = items[k & 1];
                mbar_arrive(BAR(C::B_IE + (k & 1)));
                if (!it.valid) break;
                if (it.tiles == 0) continue;
                const int two = it.n * a.G - it.i0 > 128 ? 2 : 1;
                auto issue_s = [&](int i, int pos) {
                    const uint64_t qd = sdesc_sw128(sb + i * C::Q_BYTES, 16, 1024);
                    const uint64_t kd = sdesc_sw128(sb + C::OFF_K + pos % C::NS * C::K_BYTES, 16, 1024);
#pragma unroll 2
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk >> 2) * C::SUB + (kk & 3) * 32;
                        tc_mma_ss(tmem + i * BN, sdesc_advance(qd, off), sdesc_advance(kd, off), C::IDESC_S, kk > 0);
                    }
                    tc_commit(BAR(C::B_S + i));
                };
                auto issue_pv = [&](int i, int pos, bool first) {
                    const uint64_t vd = sdesc_sw128(sb + C::OFF_V + pos % C::NS * C::V_BYTES, C::SUB, 1024);
#pragma unroll 2
                    for (int kk = 0; kk < BN / 16; ++kk)       // the weights of 64 keys lie over the first half of their scores
                        tc_mma_ts(tmem + 256 + i * 128, tmem + i * BN + kk * 8 + (kk >> 2) * 32, sdesc_advance(vd, kk * 2048), C::IDESC_PV,
                                    (!first || kk > 0) ? 1u : 0u);
                };
                if (TREE && it.alt) {
                    // key tile j on row tile j & 1, two of them under way
                    const int both = it.tiles > 1 ? 2 : 1;
                    for (int i = 0; ok && i < both; ++i) {
                        ok = wait(C::B_Q + i, seen[i], 0xE8) && wait(C::B_KF + (t + i) % C::NS, (t + i) / C::NS, 0xE9);
                        if (!ok) break;
                        tc_fence_after();
                        issue_s(i, t + i);
                        tc_commit(BAR(C::B_KE + (t + i) % C::NS));
                    }
                    for (int j = 0; ok && j < it.tiles; ++j, ++t) {
                        const int i = j & 1;
                        if (!(ok = wait(C::B_VF + t % C::NS, t / C::NS, 0xEA) && wait(C::B_P + i, np[i], 0xEB))) break;
                        if (j < 2 && seen[i] > 0 && !(ok = wait(C::B_OE + i, seen[i] - 1, 0xEC))) break;
                        ++np[i];
                        tc_fence_after();
                        issue_pv(i, t, j < 2);
                        tc_commit(BAR(C::B_VE + t % C::NS));
                        if (j + 2 >= it.tiles) tc_commit(BAR(C::B_O + i));
                        if (j + 2 < it.tiles) {
                            if (!(ok = wait(C::B_KF + t % C::NS, t / C::NS + 1, 0xED))) break;
                            tc_fence_after();
                            issue_s(i, t + 2);
                            tc_commit(BAR(C::B_KE + t % C::NS));
                        }
                    }
                    for (int i = 0; i < both; ++i) ++seen[i];
                    continue;
                }
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
                        if (i == two - 1) tc_commit(BAR(C::B_KE + t % C::NS));   // S(j) is complete
                        tc_fence_after();
                        issue_pv(i, t, j == 0);
                        if (j == it.tiles - 1) tc_commit(BAR(C::B_O + i));
                        if (j + 1 < it.tiles) {
                            if (i == 0) {
                                if (!(ok = wait(C::B_KF + (t + 1) % C::NS, (t + 1) / C::NS, 0xED))) break;
                                tc_fence_after();
                            }
                            issue_s(i, t + 1);
                        }
                    }
                    if (!ok) break;
                    tc_commit(BAR(C::B_VE + t % C::NS));
                }
                for (int i = 0; i < two; ++i) ++seen[i];
            }
            // every product issued is complete before TMEM is freed
            tc_commit(BAR(C::B_FIN));
            int never = 0;
            mbar_wait(BAR(C::B_FIN), 0, &never, a.status, 0xEE);
            }
            __syncwarp();
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
        int xs = 0;
        // All sixteen softmax warps; what each of them knows of TMEM (products complete, sums read) the others know behind it:
        // the barrier alone does not order tensor-memory accesses.
        auto meet_all = [&]() {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(C::B_X));
            const bool met = wait(C::B_X, xs++, 0xF5);
            tc_fence_after();
            return met;
        };
        int t = 0, cs = 0, seen = 0;   // key tiles, S tiles and items with work of this row tile
        bool ok = true;
        for (int k = 0; ok; ++k) {
            if (!wait(C::B_IF + (k & 1), k >> 1, 0xF0)) break;
            const Item it = items[k & 1];
            __syncwarp();
            if (lane == 0) mbar_arrive(BAR(C::B_IE + (k & 1)));
            if (!it.valid) break;
            const bool alt = TREE && it.alt;
            const int rows = it.n * a.G, ri = it.i0 + (alt ? 0 : qt * 128) + row;
            // busy: the tile has rows (and key tiles of its own)
            const bool there = ri < rows, busy = alt ? qt < it.tiles : it.i0 + qt * 128 < rows;
            const int tok = there ? ri / a.G : 0, head = it.hk * a.G + (there ? ri - tok * a.G : 0);
            int kmin = 0, kmax = INT_MAX;      // a row that is not there masks nothing (q = 0)
            TreeRow tr = {};
            if (there && TREE) {
                tr = tree_row(a, Req{it.row0, it.n, it.len, false}, tok);
                kmin = tr.lo;
                kmax = tr.ctx - 1;     // every key from kmin to kmax is seen
            } else if (there) {
                row_keys(a, Req{it.row0, it.n, it.len, false}, tok, kmin, kmax);
            }
            float f_row = 1.f;
            if (busy && it.tiles) {
                // ---- the rows of q as fp16, each one's largest value scaled into [2^7, 2^8).  Each warp of the pair takes 16
                // of the 32 rows: as they are into their places in the tile, all copies under way together (PER lanes
                // read a row), and there converted, one pass of a few rows after the other: straight code for all of
                // them, run once an item, waited 9 us for its instructions.  The pair tells each other the exponents.
                constexpr int PER = D / 8, ROWS = 32 / PER;               // lanes of a row, rows of a read
                const int64_t mine = there ? static_cast<int64_t>(it.row0 + tok) * a.qs[0] + static_cast<int64_t>(head) * a.qs[1] : -1;
                const __nv_bfloat16* const q = static_cast<const __nv_bfloat16*>(a.q);
                const int c = lane % PER, r0 = 16 * half + lane / PER;    // 16 bytes of the row, first of the warp's 32 rows
                uint8_t* const tile = smem + qt * C::Q_BYTES + (c >> 3) * C::SUB;
                const int in_tile = (warp & 3) * 32;
#pragma unroll 1
                for (int i = 0; i < 16; i += ROWS) {
                    const int64_t at = __shfl_sync(0xffffffffu, mine, r0 + i);
                    uint8_t* to = tile + sw128_offset(in_tile + r0 + i, c & 7);
                    const bool on = at >= 0 && 8 * c < a.d;
                    const __nv_bfloat16* from = q + at + 8 * c;
                    if (vec_q) {
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(to)), "l"(on ? from : q), "r"(on ? 16 : 0) : "memory");
                    } else {
                        for (int e = 0; e < 8; ++e)
                            reinterpret_cast<unsigned short*>(to)[e] = on ? reinterpret_cast<const unsigned short*>(from)[e] : static_cast<unsigned short>(0);
                    }
                }
                asm volatile("cp.async.wait_all;" ::: "memory");
                int8_t* const exps = reinterpret_cast<int8_t*>(smem + C::OFF_EXP) + 32 * pair;
#pragma unroll 1
                for (int i = 0; i < 16; i += ROWS) {
                    uint4* at = reinterpret_cast<uint4*>(tile + sw128_offset(in_tile + r0 + i, c & 7));   // this lane's own copy
                    const uint4 x = *at;
                    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                    uint32_t top = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7fff0000u, (w[e] << 16) & 0x7fff0000u));
#pragma unroll
                    for (int o = 1; o < PER; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
                    int ex = top && top < 0x7f800000u ? static_cast<int>(top >> 23) - 127 - 7 : 0;
                    ex = min(max(ex, -126), 126);
                    const float up = __uint_as_float(static_cast<uint32_t>(127 - ex) << 23);
                    uint32_t y[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = h2(__uint_as_float(w[e] << 16) * up, __uint_as_float(w[e] & 0xffff0000u) * up);
                    *at = make_uint4(y[0], y[1], y[2], y[3]);
                    if (c == 0) exps[r0 + i] = static_cast<int8_t>(ex);
                }
                if (!(ok = meet())) break;
                f_row = __uint_as_float(static_cast<uint32_t>(127 + exps[lane]) << 23);
                fence_proxy_async_smem();
                mbar_arrive(BAR(C::B_Q + qt));
            }
            float M = -INFINITY, xm = -INFINITY, L = 0.f;      // M of the row; x and L of this thread's columns
            for (int j = 0; j < it.tiles; ++j, ++t) {
                const int sl = t % kMetas, k0 = (it.first + j) * BN;
                if (!(ok = wait(C::B_MF + sl, t / kMetas, 0xF1))) break;
                if (!busy || (alt && (j & 1) != qt)) {     // nothing of this row tile's: only the record's turn
                    if (lane == 0) mbar_arrive(BAR(C::B_ME + sl));
                    continue;
                }
                if (!(ok = wait(C::B_S + qt, cs, 0xF2))) break;
                ++cs;
                tc_fence_after();
                const TileMeta* mt = metas + sl;
                const bool edge = __any_sync(0xffffffffu, k0 < kmin || k0 + BN - 1 > kmax);
                constexpr int E_ON = TREE ? E_BITS : E_RANGE;
                float um, x;
                uint64_t seen_own = 0, seen_other = 0;     // of this thread's 64 keys and the other's; a row that is not there masks nothing
                if (TREE && edge) {
                    seen_own = there ? seen_from(tr, k0 + c0, it.len) : ~0ull;
                    seen_other = there ? seen_from(tr, k0 + 64 - c0, it.len) : ~0ull;
                }
                if (edge) maxima<E_ON>(tS, mt, c0, f_row, k0, kmin, kmax, seen_own, um, x);
                else maxima<E_NONE>(tS, mt, c0, f_row, k0, kmin, kmax, 0, um, x);
                xm = fmaxf(xm, x);
                const bool fresh = alt ? j < 2 : j == 0;   // the first tile of this row tile
                bool move = fresh;
                if (!move) {                   // does a row of the two warps move its M?
                    volatile int* f = flags + 2 * ((TREE ? cs : t) & 1);
                    const int mine = __any_sync(0xffffffffu, um > M + kTau);
                    if (lane == 0) f[half] = mine;
                    if (!(ok = meet())) break;
                    move = f[0] | f[1];
                }
                if (move) {                    // both threads of a row take the maximum of u over all of its columns
                    float u2, x2;
                    if (edge) maxima<E_ON>(tS, mt, 64 - c0, f_row, k0, kmin, kmax, seen_other, u2, x2);
                    else maxima<E_NONE>(tS, mt, 64 - c0, f_row, k0, kmin, kmax, 0, u2, x2);
                    um = fmaxf(um, u2);
                    float fac = 1.f;
                    // Trees: all rows that have grown move along with one that must (they share the pass over O), and
                    // M is a whole number: with scales that are powers of two lv - M is exact then (l of 131,000 keys with
                    // |x| up to 50 off by 0.87e-6 instead of 1.06e-6; the rest is the scores' sums, which are cut off).
                    const float to = TREE ? floorf(um) : um;
                    if (TREE ? to > M : um > M + kTau) {
                        fac = M == -INFINITY ? 0.f : ex2(M - to);
                        M = to;
                        L *= fac;
                    }
                    if (!fresh) {              // S(j) is complete, so every earlier W V has been added to O
#pragma unroll 1
                        for (int cc = half * (DV / 64); cc < (half + 1) * (DV / 64); ++cc) {
                            uint32_t r[32];
                            tmem_ld32(tO + cc * 32, r);
#pragma unroll
                            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * fac);
                            tmem_st32(tO + cc * 32, r);
                        }
                    }
                    tc_fence_before();
                    if (!(ok = meet())) break; // the other thread has read this one's scores, which the weights overwrite
                    tc_fence_after();
                }
                const float mref = M == -INFINITY ? 0.f : M - kOff;
                L += edge ? weights<E_ON>(tS, mt, c0, f_row, mref, k0, kmin, kmax, seen_own)
                          : weights<E_NONE>(tS, mt, c0, f_row, mref, k0, kmin, kmax, 0);
                tc_fence_before();
                mbar_arrive(BAR(C::B_P + qt));
                __syncwarp();
                if (lane == 0) mbar_arrive(BAR(C::B_ME + sl));
            }
            if (!ok) break;
            if (TREE) {
                // ---- the end of a piece: the row's sums of both half rows (alt: of both row tiles), then its columns
                if (busy && it.tiles) {
                    if (!(ok = wait(C::B_O + qt, seen, 0xF3))) break;
                    tc_fence_after();
                    ++seen;
                }
                // by way of the tiles of Q, which every product has read: [half][row] of (M, L, largest x)
                auto stat = [&](int tile) { return reinterpret_cast<float4*>(smem + tile * C::Q_BYTES) + row; };
                stat(qt)[128 * half] = make_float4(M, L, xm, 0.f);
                if (!(ok = meet_all())) break;
                const float4 s0 = stat(alt ? 0 : qt)[0], s1 = stat(alt ? 0 : qt)[128];
                float4 s2 = make_float4(-INFINITY, 0.f, -INFINITY, 0.f), s3 = s2;
                if (alt) {
                    s2 = stat(1)[0];
                    s3 = stat(1)[128];
                }
                // row tile 0 (or this one): M s0.x; with alt row tile 1: M s2.x.  Largest x of all keys, l relative to it
                float mm = fmaxf(fmaxf(s0.z, s1.z), fmaxf(s2.z, s3.z));
                const float ref = mm == -INFINITY ? 0.f : mm, La = s0.y + s1.y, Lb = s2.y + s3.y;
                auto times = [&](float x, float Mx, float lv) { return Mx == -INFINITY ? (x != x ? x : 0.f) : x * ex2(Mx - ref - lv - kOff); };
                float l = times(La, s0.x, it.lv0) + times(Lb, s2.x, it.lv0), norm = 1.f;
                const int64_t out_row = it.row0 + tok;
                const bool leads = there && half == 0 && (!alt || qt == 0), whole = it.slot < 0;
                if (!whole) {
                    if (leads) pieces.ml[static_cast<int64_t>(it.slot) * kRows + (ri - it.i0)] = make_float2(mm, l);
                } else {
                    norm = l;
                    if (a.sink) {
                        const float sk = __ldg(a.sink + head) * kLog2e, nm = fmaxf(mm, sk);
                        const float f = mm == -INFINITY ? 1.f : ex2(mm - nm);
                        l = l * f + ex2(sk - (nm == -INFINITY ? 0.f : nm));
                        norm = f == 0.f ? INFINITY : l / f;
                        mm = nm;
                    }
                    if (leads && a.m) {
                        a.m[static_cast<int64_t>(head) * a.T + out_row] = mm == -INFINITY ? mm : mm * kLn2;
                        a.l[static_cast<int64_t>(head) * a.T + out_row] = l;
                    }
                    norm = norm == 0.f ? 0.f : 1.f / norm;
                }
                // O of a row tile times 2^(M - kOff - ref) / l; NaN among the weights stays
                auto factor = [&](float Lx, float Mx) { return Mx == -INFINITY ? (Lx != Lx ? Lx : 0.f) : ex2(Mx - ref - kOff) * norm; };
                const float fa = factor(La, s0.x), fb = factor(Lb, s2.x);
                const bool hasA = it.tiles > 0, hasB = alt && it.tiles > 1;
                const uint32_t tA = alt ? tmem + 256 + lanes : tO, tB = tmem + 384 + lanes;
                __nv_bfloat16* o = static_cast<__nv_bfloat16*>(a.o) + out_row * a.os[0] + static_cast<int64_t>(head) * a.os[1];
                // four channels of all rows together: a warp's rows are written side by side
                const bool wide_o = vec_o && ((reinterpret_cast<uintptr_t>(a.o) | 2 * a.os[0] | 2 * a.os[1]) & 31) == 0;   // 32 bytes at a time
                float* part = pieces.part + static_cast<int64_t>(whole ? 0 : it.slot) * kRows * DV + 4 * (ri - it.i0);
                // 32 columns at a time: two threads to a row, four with alt
#pragma unroll 1
                for (int cc = alt ? 2 * qt + half : half; cc < DV / 32; cc += alt ? 4 : 2) {
                    float x[32];
                    uint32_t u[32];
#pragma unroll
                    for (int i = 0; i < 32; ++i) x[i] = 0.f;
                    if (hasA) {
                        tmem_ld32(tA + cc * 32, u);
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(u[i]) * fa;
                    }
                    if (hasB) {
                        tmem_ld32(tB + cc * 32, u);
#pragma unroll
                        for (int i = 0; i < 32; ++i) x[i] = fmaf(__uint_as_float(u[i]), fb, x[i]);
                    }
                    if (!there) continue;
                    if (whole && wide_o && cc * 32 + 32 <= a.dv) {
                        uint32_t w[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) w[i] = pack_bf16(x[2 * i], x[2 * i + 1]);
                        st_global_v8(o + cc * 32, w);
                        st_global_v8(o + cc * 32 + 16, w + 8);
                        continue;
                    }
                    if (!whole) {
#pragma unroll
                        for (int i = 0; i < 32; i += 4)
                            *reinterpret_cast<float4*>(part + (cc * 32 + i) * kRows) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
                        continue;
                    }
#pragma unroll
                    for (int v = 0; v < 4; ++v) {
                        if (cc * 32 + 8 * v >= a.dv) continue;
                        uint32_t w[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e) w[e] = pack_bf16(x[8 * v + 2 * e], x[8 * v + 2 * e + 1]);
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
                if (!(ok = meet_all())) break;             // the sums and both O have been read
                if (busy && it.tiles) {
                    tc_fence_before();                     // for the reads of the other row tile's warps too
                    mbar_arrive(BAR(C::B_OE + qt));
                }
                continue;
            }
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

template <int D, int DV, bool TREE>
cudaError_t launch(const CacheAttnArgs& a, const CUtensorMap* maps, uint32_t* counter, uint32_t* far, const Pieces& pieces, int most,
                   cudaStream_t s) {
    using C = Cfg<D, DV>;
    auto kernel = k_cache_attn_tc<D, DV, TREE>;
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t{1} << (dev & 63);
    if (!(done.load(std::memory_order_relaxed) & bit)) {
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM)) != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    const bool vec_q = (reinterpret_cast<uintptr_t>(a.q) & 15) == 0 && a.qs[0] % 8 == 0 && a.qs[1] % 8 == 0;
    const bool vec_o = (reinterpret_cast<uintptr_t>(a.o) & 15) == 0 && a.os[0] % 8 == 0 && a.os[1] % 8 == 0;
    kernel<<<static_cast<unsigned>(most), kThreads, C::SMEM, s>>>(maps[0], maps[1], a, counter, far, vec_q, vec_o, pieces);
    return cudaGetLastError();
}

int sms() {
    static std::atomic<int> cached[64];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
    n = cached[dev].load(std::memory_order_relaxed);
    if (n > 0) return n;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n < 1) return 1;
    cached[dev].store(n, std::memory_order_relaxed);
    return n;
}

// CTAs of a call: trees, one per SM; else no more than the packed rows' groups and a ragged one per request.
int ctas_of(const CacheAttnArgs& a) {
    const int64_t most = (static_cast<int64_t>(a.T) * a.G / kRows + a.R) * a.Hkv;
    return a.tree ? std::min(sms(), kMaxTcCtas) : static_cast<int>(std::min<int64_t>(sms(), most));
}

}  // namespace

size_t cache_attn_tc_workspace(const CacheAttnArgs& a) {
    if (!a.tree || !cache_attn_tc_takes(a)) return 0;
    const size_t slots = 2 * static_cast<size_t>(kMaxTcCtas) * kRows, DV = a.dv <= 64 ? 64 : 128;
    return (sizeof(Rec) * kMaxTcCtas + 255) / 256 * 256 + slots * sizeof(float2) + slots * DV * sizeof(float);
}

bool cache_attn_tc_takes(const CacheAttnArgs& a) {
    if (a.dtype != BPA_BF16 || a.d % 16 || a.dv % 16 || a.d > 128 || a.dv > 128 || (a.d <= 64 && a.dv > 64) || a.P % 16) return false;
    const int64_t rows = static_cast<int64_t>(a.max_q) * a.G;
    if (rows <= (a.tree ? kFewTreeRows : kFewRows)) return false;
    if (a.tree) {
        // Items are cut between CTAs, so the rows may be few; what counts is the work, in products of 64 rows with 128
        // keys of 256 channels.  Measured (this kernel and the other one alone, us, 4 q heads on each of 8 kv heads,
        // 128 + 128 channels): 104 rows a request, 416 of them 32.8 and 34.9, 36.9 and 34.6, 832 35.9 and 46.0; 256 rows, 512 of
        // them 38.9 and 37.5, 1,024 41.0 and 51.4; but 40 and 60 rows, which leave most of a row tile of 128 empty, 660
        // 52.0 and 47.9, 990 59.3 and 55.4, 1,320 72.4 and 78.5, 1,980 73.5 and 81.8; 33 requests of 8 to 120 rows, window 1,024,
        // 64 + 64 channels, 1,215 of them 80.6 and 75.5.  The keys are those that the page table has room for (the lengths are
        // on the device), here as many as there are.  With room for 131,072 tokens every step of more than kFewTreeRows rows
        // comes here: 8 requests of 8 to 16 rows over 200 to 2,000 tokens 55.7 us instead of 42.3, 32 over 100 to 500 tokens
        // 67.9 instead of 52.8, one of 26 rows over 1,500 tokens 37.9 instead of 36.0; larger ones come here anyway.
        int64_t keys = static_cast<int64_t>(a.max_pages) * a.P;
        if (a.wl >= 0) keys = std::min(keys, static_cast<int64_t>(a.wl) + a.max_q + BN);
        const double work = static_cast<double>(a.T) * a.G / 64 * a.Hkv * keys / 128 * (a.d + a.dv) / 256;
        return work >= (static_cast<int64_t>(a.T) * a.G >= 96 * static_cast<int64_t>(a.R) ? 500 : 1300);
    }
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

CacheBox cache_attn_tc_box(const CacheAttnArgs& a) { return {a.d <= 64 ? 64 : 128, a.dv <= 64 ? 64 : 128, box_rows(a.P)}; }

cudaError_t launch_cache_attn_tc(const CacheAttnArgs& a, const CUtensorMap* maps, uint32_t* counter, uint32_t* far, uint8_t* ws,
                                 Pieces* left, cudaStream_t s) {
    const int ctas = ctas_of(a);
    if (!a.tree) {
        if (a.d <= 64) return launch<64, 64, false>(a, maps, counter, far, {}, ctas, s);
        return a.dv <= 64 ? launch<128, 64, false>(a, maps, counter, far, {}, ctas, s) : launch<128, 128, false>(a, maps, counter, far, {}, ctas, s);
    }
    Pieces& p = *left;
    p.recs = reinterpret_cast<Rec*>(ws);
    p.ml = reinterpret_cast<float2*>(ws + (sizeof(Rec) * kMaxTcCtas + 255) / 256 * 256);
    p.part = reinterpret_cast<float*>(p.ml + 2 * static_cast<size_t>(kMaxTcCtas) * kRows);
    p.ctas = ctas;
    p.rows_per = kRows;
    if (a.d <= 64) return launch<64, 64, true>(a, maps, counter, far, p, ctas, s);
    return a.dv <= 64 ? launch<128, 64, true>(a, maps, counter, far, p, ctas, s) : launch<128, 128, true>(a, maps, counter, far, p, ctas, s);
}

}  // namespace bpa
