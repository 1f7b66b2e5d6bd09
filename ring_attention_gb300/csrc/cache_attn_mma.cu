// cache_attn_mma.cu - attention of few query rows over the paged 8-bit cache (generation, drafts).
//
// An item is up to 64 query rows (row = token-in-request * G + q head in the group, so every row
// reads the same keys) of one request and kv head; its keys are walked in tiles of 64.  Codes are
// exact in fp16, so both products run on fp16 matrix instructions with float32 sums, keys and
// channels on the side of 16 and query rows on the side of 8 (a group of few heads wastes little):
//   S^T = K Q^T  with each row of Q scaled by a power of two into fp16's range (bf16 rows lose
//               nothing above 2^-22 of the row's largest value; float32 rows go in as two halves);
//   z = S * (k scale of the page) * (row's scale), in log2 units; m and l from exp2(z - m), float32;
//   O^T += V^T W^T  with W = exp2(z + log2(v scale) - M + 9) in fp16, M the running maximum of
//               z + log2(v scale): the weight that a page's codes really have, so pages whose scales
//               lie far apart keep their precision.  M moves only when it grows by more than 6 (W <=
//               2^15); a weight below 2^-33 of the largest is dropped.  float32: W as two halves.
//
// Bounded by the bytes of K and V where a kv head has up to 8 rows: 64 requests of 8,192 tokens, 8 kv
// heads of 128 channels, 4 q heads each 155 us (6.9 TB/s); of 200 to 8,191 tokens 98.2 us (5.7 TB/s);
// three of 100,000 to 131,071 tokens 122 us (6.1 TB/s).  Smaller pieces cost more: 40 requests of up
// to 4,095 tokens, 16 q heads a kv head, 128 + 64 channels 49.6 us (2.7 TB/s; mostly launches,
// items' starts and ends and the hand-over of tiles, which stay without the arithmetic).
// So the CTAs are persistent and each takes an equal share of all cost of all items, whatever the
// lengths: a tile counts one, two or four where its rows take one, two or four of the warps (33
// requests of 8 to 48 rows, 41.7 us now: 45.3 against 58.8 with every tile counting one), and an item's
// start and end six more (the 40 requests above: 51.3 us; four 53.9).  A share may begin and end inside
// an item.  Pieces of items go to the workspace as (m, l, O) and a second, small launch joins them in
// ascending order, so nothing is added in an order that changes.  Per CTA one warp copies tiles by TMA
// (a page's rows at a time, swizzled) into a ring of stages and passes the page's scales beside them;
// four warps take 16 keys of a tile each, or more of the keys for a part of the rows.
//
// Layouts without bank conflicts or shuffles: channels are permuted between Q and K so that a lane's
// 16 consecutive bytes of a key feed four products, and keys (n odd: n ^ 4 within eight) so that
// V's rows are read 16 bytes at a time; pairs of V's rows are interleaved by byte permutes on the way
// to fp16, and W turns from a result into an operand by two 8 x 8 transpositions.
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
constexpr int kExtra = 6;             // what an item's start and end count for in a share
constexpr int kCost2 = 2, kCost4 = 4; // what a tile counts for whose rows take two or four of the warps, else 1
constexpr int kBatch = 8;             // tiles whose page ids and scales are fetched together (four lanes each)
constexpr float kOff = 9.f;           // log2 of the largest fp16 weight right after M moved
constexpr float kLazy = 6.f;          // M moves when it grows by more

struct Rec {                          // what a CTA leaves for the join
    int trail;                        // slot 1 holds the first of `trail` pieces of an item (0: none)
    int row0, hk, i0, nrows;          // that item
    uint32_t flags, where;            // this CTA's status
    int pad;
};
static_assert(sizeof(Rec) == 32, "record");

struct Work {
    CacheAttnArgs a;
    int rows_per, ctas;               // rows of an item, CTAs
    const uint32_t* far;              // [R] or null (BESIDE): of the requests of more than kFewRows rows only those marked here
    int vec_q, vec_o;                 // four elements of q, two of o at a time
    Rec* recs;                        // [ctas]
    float2* ml;                       // [2 ctas][rows_per] (m in log2 units, l)
    float* part;                      // [2 ctas][rows_per][DVP] relative to m
};

struct Meta {
    int key0, len, n, row0, hk, i0, flags, pad;
    float ks[4], vs[4];               // scales of the tile's four 16-key chunks
};
enum { F_FIRST = 1, F_LAST = 2, F_LEAD = 4, F_TRAIL = 8, F_END = 16 };

// CTAs of an SM: what the sums (DVP / 4 registers of a thread) and q (DP / 8) leave, both times NT
constexpr int occupancy(int DP, int DVP, int NT) {
    const int regs = NT * (DVP / 4 + DP / 8);
    return regs <= 32 ? 4 : regs <= 64 ? 3 : regs <= 96 ? 2 : 1;
}

// DP, DVP: head dims of k and v padded to 64, 128 or 256; NT: query rows of a warp / 8; SPLIT: float32
template <int DP, int DVP, int NT, bool SPLIT>
struct Cfg {
    static constexpr int RBK = DP < 128 ? DP : 128, RBV = DVP < 128 ? DVP : 128;   // bytes of a swizzled row
    static constexpr int HK = DP / RBK, HV = DVP / RBV;                            // 128-byte halves
    static constexpr int K_BYTES = kTile * DP, V_BYTES = kTile * DVP, STAGE = K_BYTES + V_BYTES;
    static constexpr bool Q_REGS = !SPLIT && NT == 1;                              // else in shared memory
    static constexpr int QF = DP / 16 * NT * 256 * (SPLIT ? 2 : 1);                // fragments of a row tile
    static constexpr int QS = Q_REGS ? 0 : QF * (NT == 1 ? 1 : 4);                 // ... of all row tiles
    static constexpr int STATE = 8 * NT * DVP, STATS = 8 * NT;                     // of a warp: floats, float4
    static constexpr int MERGE = kNW * (STATE * 4 + STATS * 16);
    static constexpr int OCC = occupancy(DP, DVP, NT);
    static constexpr int FIXED = 1024 + MERGE + 256 + QS;
    static constexpr int FIT = (233472 / OCC - 1024 - 128 - FIXED) / (STAGE + (int)sizeof(Meta));
    static constexpr int NS = FIT > 8 ? 8 : FIT;
    static constexpr int SMEM = FIXED + NS * (STAGE + (int)sizeof(Meta));
    static_assert(NS >= 2, "stages");
};

// announces bytes without arriving
BPA_DEV void mbar_expect_tx_only(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
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
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// the transpose of an 8 x 8 matrix of fp16 in fragment layout
BPA_DEV uint32_t transposed(uint32_t v) {
    uint32_t r;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}
BPA_DEV uint32_t h2(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
BPA_DEV float2 h2f(uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }
// byte offset of byte `col` of row `row` in a TMA-swizzled tile with rows of RB (64 or 128) bytes
template <int RB>
BPA_DEV uint32_t swz(int row, int col) {
    const uint32_t off = row * RB + col;
    return RB == 128 ? off ^ ((row & 7u) << 4) : off ^ (((row >> 1) & 3u) << 4);
}

BPA_DEV float ld_q(const float* p) { return __ldg(p); }
BPA_DEV float ld_q(const __nv_bfloat16* p) { return __bfloat162float(*p); }
BPA_DEV void ld_q4(const float* p, float (&v)[4]) {
    const float4 x = __ldg(reinterpret_cast<const float4*>(p));
    v[0] = x.x;
    v[1] = x.y;
    v[2] = x.z;
    v[3] = x.w;
}
BPA_DEV void ld_q4(const __nv_bfloat16* p, float (&v)[4]) {
    const uint2 x = __ldg(reinterpret_cast<const uint2*>(p));
    v[0] = __uint_as_float(x.x << 16);
    v[1] = __uint_as_float(x.x & 0xffff0000u);
    v[2] = __uint_as_float(x.y << 16);
    v[3] = __uint_as_float(x.y & 0xffff0000u);
}

// Request r; BESIDE: without rows where the kernel for many rows has taken it.  An instance of its own, since
// the check in every instance cost generation 1 to 2 % (64 requests 98.6 us with it, 97.0 without).
template <bool BESIDE>
BPA_DEV Req own_request(const Work& w, int r) {
    Req q = request_of(w.a, r);
    if (BESIDE && q.n * w.a.G > kFewRows && !w.far[r]) q.n = 0;
    return q;
}

// Key tiles of row group rg: first tile and count (at least one, so that rows without keys are
// written too; such a tile holds no allowed key).
struct Tiles {
    int first, n;
    int each;                          // what a tile counts for
    BPA_DEV int cost() const { return n * each + kExtra; }
    // tiles that end within the first `c` of the cost (a tile is the share's that holds its last part)
    BPA_DEV int within(long long c) const { return c <= kExtra ? 0 : (static_cast<int>(c) - kExtra) / each; }
};
template <int NT>
BPA_DEV Tiles tiles_of(const CacheAttnArgs& a, const Req& q, int rg, int rows_per) {
    const int i0 = rg * rows_per, i1 = min(q.n * a.G, i0 + rows_per) - 1, rows = i1 - i0 + 1;
    const int each = rows <= 8 * NT ? 1 : rows <= 16 * NT ? kCost2 : kCost4;
    int lo, hi, x;
    row_keys(a, q, i0 / a.G, lo, x);
    row_keys(a, q, i1 / a.G, x, hi);
    if (lo > hi) return {0, 1, each};
    return {lo / kTile, hi / kTile - lo / kTile + 1, each};
}
template <int NT>
BPA_DEV long long cost_of_request(const CacheAttnArgs& a, const Req& q, int rows_per) {
    if (q.n == 0) return 0;
    long long n = 0;
    const int groups = (q.n * a.G + rows_per - 1) / rows_per;
    for (int rg = 0; rg < groups; ++rg) n += tiles_of<NT>(a, q, rg, rows_per).cost();
    return n * a.Hkv;
}

// total * c / parts, in 32 bits where they hold the product
BPA_DEV long long share(long long total, int c, int parts) {
    const unsigned long long x = static_cast<unsigned long long>(total) * c;
    return x >> 32 ? x / parts : static_cast<uint32_t>(x) / static_cast<uint32_t>(parts);
}

template <int DP, int DVP, int NT, bool SPLIT, bool BESIDE>
__global__ void __launch_bounds__(kThreads, (Cfg<DP, DVP, NT, SPLIT>::OCC))
    k_cache_attn_mma(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV, const Work w) {
    using C = Cfg<DP, DVP, NT, SPLIT>;
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
    const int rows_per = w.rows_per;
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
    }
    if (threadIdx.x == 32 * kNW) {
        tma_prefetch(&tmK);
        tma_prefetch(&tmV);
    }
    wait_for_previous();               // nothing of the caller's is read or written before
    if (threadIdx.x == 0) rec->flags = rec->where = 0;

    // ---- this CTA's share: [begin, end) of the running sum of the items' costs
    const int per = (a.R + kThreads - 1) / kThreads, r0 = min(a.R, static_cast<int>(threadIdx.x) * per),
              r1 = min(a.R, r0 + per);
    long long mine = 0;
    for (int r = r0; r < r1; ++r) mine += cost_of_request<NT>(a, own_request<BESIDE>(w, r), rows_per);
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
    // a share is at least a tile among the CTAs that take part, so the pieces of an item lie side by side
    const int most = rows_per <= 8 * NT ? 1 : rows_per <= 16 * NT ? kCost2 : kCost4;
    const int parts = static_cast<int>(min(total / most, static_cast<long long>(w.ctas)));
    const long long begin = cta < parts ? share(total, cta, parts) : total, end = cta < parts ? share(total, cta + 1, parts) : total;
    if (begin < end && begin >= before && begin < before + mine) {
        long long at = before;
        for (int r = r0; r < r1; ++r) {
            const long long n = cost_of_request<NT>(a, own_request<BESIDE>(w, r), rows_per);
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
        // ---- producer: the share's segments (its part of an item) in batches of up to kBatch tiles.  A
        // batch's page ids are asked for one batch ahead and its scales half a batch ahead.
        struct Batch {
            int cnt, key0, len, n, row0, hk, i0, flags;   // flags: kind; F_FIRST / F_LAST of its first / last tile
            int id;                                       // lane 4 t + c: page of chunk c of tile t (-1: none)
            float ks, vs;                                 // ... and its scales
        };
        int r = s_r, stage = 0, hk = 0, rg = 0, groups = 0, t = 0, te = 0, kind = 0;
        uint32_t phase = 1;            // the ring starts empty
        long long left = r >= 0 ? end - begin : 0, off = s_off, at = begin;   // of the cost; `at`: the running sum at `off`
        bool first = false, started = false, ok = true;
        Req rq = {};
        Tiles tl = {};
        Rec out = {};
        if (r >= 0) {
            rq = own_request<BESIDE>(w, r);
            if (rq.bad && lane == 0) report(status, ST_CHECK, 0xCD1);
            groups = (rq.n * a.G + rows_per - 1) / rows_per;
            const long long per_head = cost_of_request<NT>(a, rq, rows_per) / a.Hkv;
            hk = static_cast<int>(off / per_head);
            off -= hk * per_head;
            tl = tiles_of<NT>(a, rq, 0, rows_per);
            while (off >= tl.cost()) {
                off -= tl.cost();
                tl = tiles_of<NT>(a, rq, ++rg, rows_per);
            }
        }
        const int chunk = lane & 3;
        auto next_batch = [&](Batch& b) {
            b.cnt = 0;
            b.id = -1;
            while (t >= te) {
                if (left <= 0) return;
                if (started) {         // the next item: row group, head, request
                    if (++rg == groups) {
                        rg = 0;
                        if (++hk == a.Hkv) {
                            hk = 0;
                            do {
                                if (++r >= a.R) break;      // only if the lengths changed during the call
                                rq = own_request<BESIDE>(w, r);
                                if (rq.bad && rq.n && lane == 0) report(status, ST_CHECK, 0xCD1);
                            } while (rq.n == 0);
                            if (r >= a.R) {
                                if (lane == 0) report(status, ST_CHECK, 0xCD5);
                                left = 0;
                                return;
                            }
                            groups = (rq.n * a.G + rows_per - 1) / rows_per;
                        }
                    }
                    tl = tiles_of<NT>(a, rq, rg, rows_per);
                }
                started = true;
                // [off, to) of the item's cost; its first kExtra are no tiles
                const long long to = min(static_cast<long long>(tl.cost()), off + left);
                t = tl.within(off);
                te = tl.within(to);
                const bool lead = t > 0, trail = te < tl.n;
                kind = lead ? F_LEAD : trail ? F_TRAIL : 0;
                first = true;
                const int i0 = rg * rows_per, rows = min(rq.n * a.G - i0, rows_per);
                if (t < te) {
                    if (trail && !lead) {
                        // its pieces: up to the last CTA c with total c / parts < the end of the item's cost
                        const long long at_end = at + (tl.cost() - off);
                        out.trail = static_cast<int>((at_end * parts + total - 1) / total) - cta;
                        out.row0 = rq.row0;
                        out.hk = hk;
                        out.i0 = i0;
                        out.nrows = rows;
                    }
                    const int lines = (a.d * static_cast<int>(sizeof(E)) + 127) / 128;   // q on its way to L2
                    for (int i = lane; i < rows * lines; i += 32) {
                        const int ri = i0 + i / lines, tok = ri / a.G;
                        const E* q = static_cast<const E*>(a.q) + static_cast<int64_t>(rq.row0 + tok) * a.qs[0] +
                                     static_cast<int64_t>(hk * a.G + ri - tok * a.G) * a.qs[1];
                        asm volatile("prefetch.global.L2 [%0];" ::"l"(reinterpret_cast<const uint8_t*>(q) + 128 * (i % lines)));
                    }
                }
                left -= to - off;
                at += to - off;
                off = 0;
            }
            b.cnt = min(kBatch, te - t);
            b.key0 = (tl.first + t) * kTile;
            b.len = rq.len;
            b.n = rq.n;
            b.row0 = rq.row0;
            b.hk = hk;
            b.i0 = rg * rows_per;
            t += b.cnt;
            b.flags = kind | (first ? F_FIRST : 0) | (t == te ? F_LAST : 0);
            first = false;
            const int key = b.key0 + 16 * lane;
            if ((lane >> 2) < b.cnt && key < b.len) {
                b.id = a.table[static_cast<int64_t>(r) * a.max_pages + key / a.P];
                if (b.id < 0) b.id = -2;
            }
        };
        auto checked = [&](Batch& b) {             // ids outside the cache: reported, not copied
            if (b.id == -2 || b.id >= a.num_pages) {
                report(status, ST_CHECK, 0xCD0);
                b.id = -1;
            }
        };
        auto fetch_scales = [&](Batch& b) {
            checked(b);
            b.ks = b.vs = 0.f;
            if (b.id >= 0) {
                b.ks = a.kscale[static_cast<int64_t>(b.id) * a.Hkv + b.hk];
                b.vs = a.vscale[static_cast<int64_t>(b.id) * a.Hkv + b.hk];
            }
        };
        const int BR = min(a.P, kTile);
        const uint32_t copy = static_cast<uint32_t>(BR) * (DP + DVP);
        auto copy_tile = [&](const Batch& b, int jj, int st) {   // tile jj of the batch into stage st
            const bool copies = (lane >> 2) == jj && b.id >= 0 && (16 * chunk) % BR == 0;
            const uint32_t n = __popc(__ballot_sync(0xffffffffu, copies));
            if (lane == 0) mbar_expect_tx_only(FULL(st), n * copy);
            __syncwarp();
            if (copies) {
                const uint32_t to_k = sb + st * C::STAGE + 16 * chunk * C::RBK;
                const uint32_t to_v = sb + st * C::STAGE + C::K_BYTES + 16 * chunk * C::RBV;
                const int tok = (b.key0 + 16 * lane) % a.P;
                for (int h = 0; h < C::HK; ++h) tma_load_4d(to_k + h * kTile * C::RBK, &tmK, FULL(st), 128 * h, tok, b.hk, b.id);
                for (int h = 0; h < C::HV; ++h) tma_load_4d(to_v + h * kTile * C::RBV, &tmV, FULL(st), 128 * h, tok, b.hk, b.id);
            }
        };
        Batch cur, nxt;
        next_batch(cur);
        checked(cur);
        // the first tiles are on their way before their pages' scales are here
        int ahead = 0;
        for (; ahead < min(cur.cnt, C::NS); ++ahead) copy_tile(cur, ahead, ahead);
        fetch_scales(cur);
        next_batch(nxt);
        while (cur.cnt && ok) {
            for (int jj = 0; jj < cur.cnt; ++jj) {
                if (jj == cur.cnt / 2) fetch_scales(nxt);
                if (jj >= ahead) {
                    ok = mbar_wait(EMPTY(stage), phase, const_cast<volatile int*>(&s_abort), status, 0xCD2);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    copy_tile(cur, jj, stage);
                }
                Meta* m = meta + stage;
                if (lane == 0) {
                    m->key0 = cur.key0 + jj * kTile;
                    m->len = cur.len;
                    m->n = cur.n;
                    m->row0 = cur.row0;
                    m->hk = cur.hk;
                    m->i0 = cur.i0;
                    m->flags = (cur.flags & (F_LEAD | F_TRAIL)) | (jj == 0 ? cur.flags & F_FIRST : 0) |
                               (jj == cur.cnt - 1 ? cur.flags & F_LAST : 0);
                }
                if ((lane >> 2) == jj) {
                    m->ks[chunk] = cur.ks;
                    m->vs[chunk] = cur.vs;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(FULL(stage));
                if (++stage == C::NS) {
                    stage = 0;
                    phase ^= 1;
                }
            }
            ahead = 0;
            cur = nxt;
            next_batch(nxt);
        }
        if (ok) {                          // one more stage, without a tile: the end
            ok = __all_sync(0xffffffffu, mbar_wait(EMPTY(stage), phase, const_cast<volatile int*>(&s_abort), status, 0xCD2));
            if (ok && lane == 0) {
                meta[stage].flags = F_END;
                mbar_arrive(FULL(stage));
            }
        }
        // the copies in flight end before the CTA does: the consumers wait for them, and after a timeout
        // this warp (stages before `stage` hold this pass over the ring, the others the last one)
        if (!ok) {
            int never = 0;
            for (int s = 0; s < C::NS; ++s) mbar_wait(FULL(s), s < stage ? phase ^ 1 : phase, &never, status, 0xCD3);
        }
        if (lane == 0) {
            rec->trail = out.trail;
            rec->row0 = out.row0;
            rec->hk = out.hk;
            rec->i0 = out.i0;
            rec->nrows = out.nrows;
        }
        return;
    }

    // ---- consumers
    int rt = 0, slices = kNW, slice = warp;        // row tile of the item, warps that share its keys, this one
    const int g = lane >> 2, j = lane & 3;
    uint8_t* my_q = nullptr;
    uint32_t qf[C::Q_REGS ? DP / 16 : 1][NT][2];
    float acc[DVP / 16][NT][4];
    // rows 2j + e of n-tile nt: running (m, l) of this lane's keys, M of the row, its factor and keys
    float m[NT][2], l[NT][2], M[NT][2], f[NT][2];
    int lo[NT][2], hi[NT][2], in_lo = 0, in_hi = 0, any_lo = 0, any_hi = 0;
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
    for (;;) {
        if (!__all_sync(0xffffffffu, mbar_wait(FULL(stage), phase, const_cast<volatile int*>(&s_abort), status, 0xCD4))) return;
        const Meta* mt = meta + stage;
        const int flags = mt->flags, key0 = mt->key0, len = mt->len;
        if (flags & F_END) return;
        if (flags & F_FIRST) {
            // ---- a new item: this warp's rows of q as fp16 fragments, scaled by a power of two
            const Req rq = {mt->row0, mt->n, len, false};
            const int hk = mt->hk, nr = rq.n * a.G;
            // as many row tiles as this item has: 1, 2 or 4 of the warps apart, the others on other keys
            const int tiles = (min(nr - mt->i0, rows_per) + 8 * NT - 1) / (8 * NT), RT = tiles > 2 ? 4 : tiles;
            rt = warp & (RT - 1);
            slices = kNW / RT;
            slice = warp / RT;
            my_q = smem + (q_at - sb) + rt * C::QF + lane * 8;
            const int first = mt->i0 + rt * 8 * NT;
            in_lo = any_hi = 0;
            in_hi = any_lo = INT_MAX;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int ri = first + 8 * nt + g;          // the row whose channels this lane loads
                const bool there = ri < nr;
                const int tok = there ? ri / a.G : 0;
                const E* q = static_cast<const E*>(a.q) + static_cast<int64_t>(rq.row0 + tok) * a.qs[0] +
                             static_cast<int64_t>(hk * a.G + (there ? ri - tok * a.G : 0)) * a.qs[1];
                float v[DP / 16][4];
                float top = 0.f;
                if (w.vec_q) {
#pragma unroll
                    for (int s = 0; s < DP / 16; ++s) {
                        const int c = (s >> 2) * 64 + 16 * j + 4 * (s & 3);
                        v[s][0] = v[s][1] = v[s][2] = v[s][3] = 0.f;
                        if (there && c < a.d) ld_q4(q + c, v[s]);
                    }
                } else {
#pragma unroll
                    for (int s = 0; s < DP / 16; ++s) {
                        const int c = (s >> 2) * 64 + 16 * j + 4 * (s & 3);
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[s][e] = there && c < a.d ? ld_q(q + c + e) : 0.f;
                    }
                }
#pragma unroll
                for (int s = 0; s < DP / 16; ++s)
                    top = fmaxf(fmaxf(top, fmaxf(fabsf(v[s][0]), fabsf(v[s][1]))), fmaxf(fabsf(v[s][2]), fabsf(v[s][3])));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                // largest value into [2^7, 2^8); 0 and values that are not finite stay as they are
                int x = top > 0.f && top < INFINITY ? static_cast<int>(__float_as_uint(top) >> 23) - 127 - 7 : 0;
                x = min(max(x, -126), 126);
                const float up = __uint_as_float(static_cast<uint32_t>(127 - x) << 23);
                const float fac = __uint_as_float(static_cast<uint32_t>(127 + x) << 23) * a.scale * kLog2e;
#pragma unroll
                for (int s = 0; s < DP / 16; ++s) {
                    const float x0 = v[s][0] * up, x1 = v[s][1] * up, x2 = v[s][2] * up, x3 = v[s][3] * up;
                    const uint32_t p0 = h2(x0, x1), p1 = h2(x2, x3);
                    if constexpr (C::Q_REGS) {
                        qf[s][nt][0] = p0;
                        qf[s][nt][1] = p1;
                    } else {
                        uint2* at = reinterpret_cast<uint2*>(my_q + (s * NT + nt) * 256 * (SPLIT ? 2 : 1));
                        at[0] = make_uint2(p0, p1);
                        if (SPLIT) {
                            const float2 y0 = h2f(p0), y1 = h2f(p1);
                            at[32] = make_uint2(h2(x0 - y0.x, x1 - y0.y), h2(x2 - y1.x, x3 - y1.y));
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    f[nt][e] = __shfl_sync(0xffffffffu, fac, (2 * j + e) * 4);
                    const int r2 = first + 8 * nt + 2 * j + e;
                    lo[nt][e] = 0;                           // a row that is not there masks nothing (z = 0)
                    hi[nt][e] = INT_MAX;
                    if (r2 < nr) {
                        row_keys(a, rq, r2 / a.G, lo[nt][e], hi[nt][e]);
                        any_lo = min(any_lo, lo[nt][e]);
                        any_hi = max(any_hi, hi[nt][e]);
                    }
                    in_lo = max(in_lo, lo[nt][e]);           // keys that no row masks, keys that some row allows
                    in_hi = min(in_hi, hi[nt][e]);
                    m[nt][e] = M[nt][e] = -INFINITY;
                    l[nt][e] = 0.f;
                }
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                in_lo = max(in_lo, __shfl_xor_sync(0xffffffffu, in_lo, o));
                in_hi = min(in_hi, __shfl_xor_sync(0xffffffffu, in_hi, o));
                any_lo = min(any_lo, __shfl_xor_sync(0xffffffffu, any_lo, o));
                any_hi = max(any_hi, __shfl_xor_sync(0xffffffffu, any_hi, o));
            }
            any_hi = first < nr ? min(any_hi, len - 1) : -1;
            in_hi = min(in_hi, len - 1);
#pragma unroll
            for (int i = 0; i < DVP / 16; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) acc[i][nt][0] = acc[i][nt][1] = acc[i][nt][2] = acc[i][nt][3] = 0.f;
            __syncwarp();
        }
        const uint8_t *kt = smem + stage * C::STAGE, *vt = kt + C::K_BYTES;
        for (int ch = slice; ch < 4; ch += slices) {
            const int base = key0 + 16 * ch;
            if (base > any_hi || base + 15 < any_lo) continue;
            // ---- S^T = K Q^T for 16 keys: row r of a fragment is key r (even) or r ^ 4 (odd) of its eight
            const int kr = (g & 1) ? (g ^ 4) : g;
            float s[NT][2][4];
#pragma unroll
            for (int i = 0; i < 8 * NT; ++i) (&s[0][0][0])[i] = 0.f;
#pragma unroll
            for (int kk = 0; kk < DP / 64; ++kk) {
                const uint8_t* kp = kt + (kk >> 1) * kTile * C::RBK;
                const uint4 ka = *reinterpret_cast<const uint4*>(kp + swz<C::RBK>(16 * ch + kr, (kk & 1) * 64 + 16 * j));
                const uint4 kb = *reinterpret_cast<const uint4*>(kp + swz<C::RBK>(16 * ch + 8 + kr, (kk & 1) * 64 + 16 * j));
                const uint32_t wa[4] = {ka.x, ka.y, ka.z, ka.w}, wb[4] = {kb.x, kb.y, kb.z, kb.w};
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint32_t fr[4] = {cvt2(wa[u]), cvt2(wb[u]), cvt2_hi(wa[u]), cvt2_hi(wb[u])};
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        if constexpr (C::Q_REGS) {
                            mma(s[nt][u & 1], fr, qf[kk * 4 + u][nt][0], qf[kk * 4 + u][nt][1]);
                        } else {
                            const uint2* at = reinterpret_cast<const uint2*>(my_q + ((kk * 4 + u) * NT + nt) * 256 * (SPLIT ? 2 : 1));
                            const uint2 qa = at[0];
                            mma(s[nt][u & 1], fr, qa.x, qa.y);
                            if (SPLIT) {
                                const uint2 qb = at[32];
                                mma(s[nt][u & 1], fr, qb.x, qb.y);
                            }
                        }
                    }
                }
            }
            // ---- scores; z[nt][e], z[nt][2 + e]: row 2j + e, keys kr and 8 + kr
            const float ks = mt->ks[ch], vs = mt->vs[ch];
            const bool edge = base < in_lo || base + 15 > in_hi;
            const float lv = __log2f(vs);
            float z[NT][4], u[NT][2];
            bool move = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const float fk = f[nt][e] * ks;
                    float z0 = (s[nt][0][e] + s[nt][1][e]) * fk, z1 = (s[nt][0][2 + e] + s[nt][1][2 + e]) * fk;
                    if (edge) {
                        const int k0 = base + kr, k1 = base + 8 + kr;
                        if (k0 >= len || k0 < lo[nt][e] || k0 > hi[nt][e]) z0 = -INFINITY;
                        if (k1 >= len || k1 < lo[nt][e] || k1 > hi[nt][e]) z1 = -INFINITY;
                    }
                    z[nt][e] = z0;
                    z[nt][2 + e] = z1;
                    // m, l of this lane's keys (the row's eight lanes are joined at the end of the item)
                    const float c = fmaxf(z0, z1), n = fmaxf(m[nt][e], c), ref = n == -INFINITY ? 0.f : n;
                    l[nt][e] = l[nt][e] * ex2(m[nt][e] - ref) + (ex2(z0 - ref) + ex2(z1 - ref));
                    m[nt][e] = n;
                    u[nt][e] = c + lv;
                    move |= u[nt][e] > M[nt][e] + kLazy;
                }
            }
            // ---- weights in fp16, relative to M
            if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float x[2];
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
#pragma unroll
                        for (int o = 4; o < 32; o <<= 1) u[nt][e] = fmaxf(u[nt][e], __shfl_xor_sync(0xffffffffu, u[nt][e], o));
                        const float N = fmaxf(M[nt][e], u[nt][e]);
                        x[e] = M[nt][e] == -INFINITY ? 0.f : ex2(M[nt][e] - N);
                        M[nt][e] = N;
                    }
#pragma unroll
                    for (int i = 0; i < DVP / 16; ++i) {
                        acc[i][nt][0] *= x[0];
                        acc[i][nt][1] *= x[1];
                        acc[i][nt][2] *= x[0];
                        acc[i][nt][3] *= x[1];
                    }
                }
            }
            uint32_t wf[NT][2], wl[NT][2];
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                // a page of scale 0 has lv = -inf and so weights of 0, as has a row without a key so far; the
                // product is taken all the same, for codes that stand for NaN (0 * NaN)
                const float t0 = (M[nt][0] == -INFINITY ? INFINITY : M[nt][0] - lv) - kOff;
                const float t1 = (M[nt][1] == -INFINITY ? INFINITY : M[nt][1] - lv) - kOff;
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float y0 = ex2(z[nt][2 * k] - t0), y1 = ex2(z[nt][2 * k + 1] - t1);
                    const uint32_t hh = h2(y0, y1);
                    wf[nt][k] = transposed(hh);
                    if (SPLIT) {
                        const float2 r = h2f(hh);
                        wl[nt][k] = transposed(h2(y0 - r.x, y1 - r.y));
                    }
                }
            }
            // ---- O^T += V^T W^T: this lane's four keys, CV consecutive channels (two rows of a fragment each)
            constexpr int CV = (DVP < 128 ? DVP : 128) / 8;          // 8 or 16
            const int key[4] = {2 * j, (2 * j + 1) ^ 4, 8 + 2 * j, 8 + ((2 * j + 1) ^ 4)};
#pragma unroll
            for (int hv = 0; hv < C::HV; ++hv) {
                uint32_t v[4][CV / 4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint8_t* at = vt + hv * kTile * C::RBV + swz<C::RBV>(16 * ch + key[i], CV * g);
                    if constexpr (CV == 16) {
                        const uint4 x4 = *reinterpret_cast<const uint4*>(at);
                        v[i][0] = x4.x;
                        v[i][1] = x4.y;
                        v[i][2] = x4.z;
                        v[i][3] = x4.w;
                    } else {
                        const uint2 x2 = *reinterpret_cast<const uint2*>(at);
                        v[i][0] = x2.x;
                        v[i][1] = x2.y;
                    }
                }
                if (base + 16 > len) {
                    // slots past the last token may hold anything: their weight is 0, NaN is not
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if (base + key[i] >= len)
#pragma unroll
                            for (int c = 0; c < CV / 4; ++c) v[i][c] = 0;
                }
#pragma unroll
                for (int c = 0; c < CV / 4; ++c) {
                    const uint32_t ab0 = __byte_perm(v[0][c], v[1][c], 0x5140), ab1 = __byte_perm(v[0][c], v[1][c], 0x7362);
                    const uint32_t cd0 = __byte_perm(v[2][c], v[3][c], 0x5140), cd1 = __byte_perm(v[2][c], v[3][c], 0x7362);
                    const uint32_t fa[4] = {cvt2(ab0), cvt2_hi(ab0), cvt2(cd0), cvt2_hi(cd0)};
                    const uint32_t fb[4] = {cvt2(ab1), cvt2_hi(ab1), cvt2(cd1), cvt2_hi(cd1)};
                    const int i = hv * (CV / 2) + 2 * c;
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) {
                        mma(acc[i][nt], fa, wf[nt][0], wf[nt][1]);
                        mma(acc[i + 1][nt], fb, wf[nt][0], wf[nt][1]);
                        if (SPLIT) {
                            mma(acc[i][nt], fa, wl[nt][0], wl[nt][1]);
                            mma(acc[i + 1][nt], fb, wl[nt][0], wl[nt][1]);
                        }
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

        // ---- the end of this CTA's share of the item: join the lanes, then the warps' slices, in a fixed order
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int e = 0; e < 2; ++e)
#pragma unroll
                for (int o = 4; o < 32; o <<= 1) {
                    const float x = __shfl_xor_sync(0xffffffffu, m[nt][e], o), y = __shfl_xor_sync(0xffffffffu, l[nt][e], o);
                    const float n = fmaxf(m[nt][e], x), ref = n == -INFINITY ? 0.f : n;
                    // the same sum on both lanes, whichever is which
                    l[nt][e] = __fadd_rn(__fmul_rn(l[nt][e], ex2(m[nt][e] - ref)), __fmul_rn(y, ex2(x - ref)));
                    m[nt][e] = n;
                }
        // Each warp's (m, l, M) and sums go to shared memory; a thread per row turns them into the
        // slices' factors, then all threads add the slices up (every warp working out its rows' factors
        // itself, with one meeting less: 51.6 us against 50.7 for the 40 requests above).
        constexpr int CV = (DVP < 128 ? DVP : 128) / 8, F = DVP / 16;
        const int RT = kNW / slices, rows = min(nr - i0, RT * C::STATS);
        float4* stats = reinterpret_cast<float4*>(merge + kNW * C::STATE);   // [slice][row of the item]
        if (g == 0)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    stats[warp * C::STATS + 8 * nt + 2 * j + e] = make_float4(m[nt][e], l[nt][e], M[nt][e], 0.f);
        float4* buf = reinterpret_cast<float4*>(merge + warp * C::STATE) + lane;
#pragma unroll
        for (int i = 0; i < F; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
                buf[(i * NT + nt) * 32] = make_float4(acc[i][nt][0], acc[i][nt][1], acc[i][nt][2], acc[i][nt][3]);
        if (!consumers_meet()) return;
        for (int row = threadIdx.x; row < rows; row += 32 * kNW) {
            const int tok = (i0 + row) / a.G, head = hk * a.G + (i0 + row) - tok * a.G;
            float mm = -INFINITY, ll = 0.f;
#pragma unroll 4
            for (int k = 0; k < slices; ++k) mm = fmaxf(mm, stats[k * RT * C::STATS + row].x);
            const float ref = mm == -INFINITY ? 0.f : mm;
#pragma unroll 4
            for (int k = 0; k < slices; ++k) {
                const float4 b = stats[k * RT * C::STATS + row];
                ll += b.y * ex2(b.x - ref);
            }
            float norm = 1.f;
            if (flags & (F_LEAD | F_TRAIL)) {
                w.ml[(2 * static_cast<int64_t>(cta) + (flags & F_TRAIL ? 1 : 0)) * rows_per + row] = make_float2(mm, ll);
            } else {
                float lf = ll, mf = mm;
                if (a.sink) {
                    const float sk = __ldg(a.sink + head) * kLog2e;
                    mf = fmaxf(mm, sk);
                    norm = mm == -INFINITY ? 1.f : ex2(mm - mf);
                    lf = ll * norm + ex2(sk - (mf == -INFINITY ? 0.f : mf));
                }
                if (a.m) {
                    a.m[static_cast<int64_t>(head) * a.T + row0 + tok] = mf == -INFINITY ? mf : mf * kLn2;
                    a.l[static_cast<int64_t>(head) * a.T + row0 + tok] = lf;
                }
                norm = lf == 0.f ? 0.f : norm / lf;
            }
#pragma unroll 4
            for (int k = 0; k < slices; ++k) {
                float4& b = stats[k * RT * C::STATS + row];
                b.w = b.z == -INFINITY ? (norm != norm ? norm : 0.f) : ex2(b.z - kOff - ref) * norm;
            }
        }
        if (!consumers_meet()) return;
        // a warp adds four channels of 2 x 4 rows a lane, in the layout in which they were stored (no bank
        // conflicts; two channels a thread in the order of the output had sixteen-fold ones)
        for (int x = warp; x < RT * NT * (F / 2); x += kNW) {
            const int tile = x / (NT * (F / 2)), y = x - tile * (NT * (F / 2)), nt = y / (F / 2), i = 2 * (y - nt * (F / 2));
            const int r0 = tile * C::STATS + 8 * nt + 2 * j;         // this lane's rows: r0, r0 + 1
            if (r0 >= rows) continue;
            const float4* at = reinterpret_cast<const float4*>(merge + tile * C::STATE) + (i * NT + nt) * 32 + lane;
            float sum[2][4] = {};
#pragma unroll 4
            for (int k = 0; k < slices; ++k) {
                const float f0 = stats[k * RT * C::STATS + r0].w, f1 = stats[k * RT * C::STATS + r0 + 1].w;
                const float4 p = at[k * RT * (C::STATE / 4)], q = at[k * RT * (C::STATE / 4) + NT * 32];
                sum[0][0] = fmaf(p.x, f0, sum[0][0]);
                sum[0][1] = fmaf(p.z, f0, sum[0][1]);
                sum[0][2] = fmaf(q.x, f0, sum[0][2]);
                sum[0][3] = fmaf(q.z, f0, sum[0][3]);
                sum[1][0] = fmaf(p.y, f1, sum[1][0]);
                sum[1][1] = fmaf(p.w, f1, sum[1][1]);
                sum[1][2] = fmaf(q.y, f1, sum[1][2]);
                sum[1][3] = fmaf(q.w, f1, sum[1][3]);
            }
            const int c = (i / (CV / 2)) * 128 + CV * g + (i % (CV / 2)) * 2;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int row = r0 + e;
                if (row >= rows) continue;
                if (flags & (F_LEAD | F_TRAIL)) {
                    const int64_t slot = (2 * static_cast<int64_t>(cta) + (flags & F_TRAIL ? 1 : 0)) * rows_per + row;
                    *reinterpret_cast<float4*>(w.part + slot * DVP + c) = make_float4(sum[e][0], sum[e][1], sum[e][2], sum[e][3]);
                } else if (c < a.dv) {
                    const int tok = (i0 + row) / a.G, head = hk * a.G + (i0 + row) - tok * a.G;
                    E* o = static_cast<E*>(a.o) + static_cast<int64_t>(row0 + tok) * a.os[0] +
                           static_cast<int64_t>(head) * a.os[1] + c;
                    if (!SPLIT && w.vec_o) {
                        reinterpret_cast<uint32_t*>(o)[0] = pack_bf16(sum[e][0], sum[e][1]);
                        reinterpret_cast<uint32_t*>(o)[1] = pack_bf16(sum[e][2], sum[e][3]);
                    } else {
#pragma unroll
                        for (int h = 0; h < 4; ++h) o[h] = static_cast<E>(sum[e][h]);
                    }
                }
            }
        }
        if (!consumers_meet()) return;                     // the buffers may be written again
    }
}

// Joins the pieces of the items that CTA boundaries cut: the block of the CTA in which an item
// begins, rpb rows of it (a warp per row and every (8 / rpb)-th piece), pieces in ascending order.
template <int DVP, typename E>
__global__ void __launch_bounds__(256) k_cache_join(const Work w, int rpb, uint32_t* out_status) {
    constexpr int V = DVP / 32;
    __shared__ float s_acc[8][DVP];
    __shared__ float2 s_ml[8];
    __shared__ uint32_t s_flags, s_where;
    const CacheAttnArgs& a = w.a;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x;
    wait_for_previous();
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
            if (!w.far) {
                out_status[0] = s_flags;
                out_status[1] = s_where;
            } else if (s_flags) {                  // beside what the other kernel has reported
                report(out_status, s_flags, s_where);
            }
        }
    }
    const Rec rec = w.recs[c];
    const int row = blockIdx.y * rpb + warp % rpb, part = warp / rpb, parts = 8 / rpb, n = rec.trail;
    if (!n || static_cast<int>(blockIdx.y) * rpb >= rec.nrows) return;
    const bool there = row < rec.nrows;
    float m = -INFINITY, l = 0.f, acc[V];
#pragma unroll
    for (int i = 0; i < V; ++i) acc[i] = 0.f;
    if (there) {
        // one pass with the running maximum; four pieces' loads at a time
        for (int k0 = part; k0 < n; k0 += 4 * parts) {
            float2 x[4];
            float v[4][V];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int k = k0 + q * parts;
                x[q] = make_float2(-INFINITY, 0.f);
                if (k >= n) continue;
                const int64_t s = (2 * (static_cast<int64_t>(c) + k) + (k == 0)) * w.rows_per + row;
                x[q] = w.ml[s];
                const float* p = w.part + s * DVP + lane * V;
                if constexpr (V == 2) {
                    const float2 t = *reinterpret_cast<const float2*>(p);
                    v[q][0] = t.x;
                    v[q][1] = t.y;
                } else {
#pragma unroll
                    for (int i = 0; i < V; i += 4) {
                        const float4 t = *reinterpret_cast<const float4*>(p + i);
                        v[q][i] = t.x;
                        v[q][i + 1] = t.y;
                        v[q][i + 2] = t.z;
                        v[q][i + 3] = t.w;
                    }
                }
            }
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if (k0 + q * parts >= n || x[q].y == 0.f) continue;      // no keys in the piece
                const float nm = fmaxf(m, x[q].x), ref = nm == -INFINITY ? 0.f : nm;
                const float f0 = m == -INFINITY ? (l != l ? l : 0.f) : ex2(m - ref), f1 = ex2(x[q].x - ref);
                l = l * f0 + x[q].y * f1;
#pragma unroll
                for (int i = 0; i < V; ++i) acc[i] = acc[i] * f0 + v[q][i] * f1;
                m = nm;
            }
        }
    }
    if (parts > 1) {                               // the groups of pieces, in order
        if (lane == 0) s_ml[warp] = make_float2(m, l);
#pragma unroll
        for (int i = 0; i < V; ++i) s_acc[warp][lane * V + i] = acc[i];
        __syncthreads();
        if (part) return;
        for (int q = 1; q < parts; ++q) {
            const float2 x = s_ml[q * rpb + warp];
            if (x.y == 0.f) continue;
            const float nm = fmaxf(m, x.x), ref = nm == -INFINITY ? 0.f : nm;
            const float f0 = m == -INFINITY ? (l != l ? l : 0.f) : ex2(m - ref), f1 = ex2(x.x - ref);
            l = l * f0 + x.y * f1;
#pragma unroll
            for (int i = 0; i < V; ++i) acc[i] = acc[i] * f0 + s_acc[q * rpb + warp][lane * V + i] * f1;
            m = nm;
        }
    }
    if (!there) return;
    const int ri = rec.i0 + row, tok = ri / a.G, head = rec.hk * a.G + ri - tok * a.G;
    float x = 1.f;
    if (a.sink) {
        const float sk = __ldg(a.sink + head) * kLog2e, nm = fmaxf(m, sk);
        x = m == -INFINITY ? 1.f : ex2(m - nm);
        l = l * x + ex2(sk - (nm == -INFINITY ? 0.f : nm));
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
constexpr size_t kFarAt = 256;        // the marks lie behind the header

struct Plan {
    int DP, DVP, NT, RT, rows_per, occ, max_ctas;
    size_t recs, ml, part, total;     // offsets in the workspace, behind the header and the marks
};
bool plan_of(const CacheAttnArgs& a, Plan& p) {
    if (a.d % 16 || a.dv % 16 || a.d > 256 || a.dv > 256) return false;
    if (static_cast<int64_t>(a.T) * a.G > int64_t{1} << 30) return false;   // a request's rows are numbered in 32 bits
    if (a.P % 16 || (a.P < kTile ? kTile % a.P : a.P % kTile)) return false;
    p.DP = a.d <= 64 ? 64 : a.d <= 128 ? 128 : 256;
    p.DVP = a.dv <= 64 ? 64 : a.dv <= 128 ? 128 : 256;
    if (p.DVP > p.DP) p.DP = p.DVP;
    if (p.DP == 256 && p.DVP == 64) p.DVP = 128;
    const int64_t rows = static_cast<int64_t>(a.max_q > 0 ? a.max_q : 1) * a.G;
    // Up to 8 rows half as many registers leave more CTAs on an SM: 98.5 us against 142 with 16 rows a warp (64
    // requests of 200 to 8,191 tokens, 4 rows a kv head).  With 16 rows one warp converts a code once: 55
    // us against 58 with two warps of 8 rows (40 of up to 4,095), and with 8 to 48 rows 45.1 against 47.0.
    // The host knows only max_q: one token of many requests beside a request of more, or with max_q
    // unknown, is computed 16 rows a warp too (98 us -> 151).
    p.NT = rows <= 8 ? 1 : 2;
    p.RT = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
    p.rows_per = 8 * p.NT * p.RT;
    p.occ = occupancy(p.DP, p.DVP, p.NT);
    p.max_ctas = kMaxSms * p.occ;
    auto up = [](size_t x) { return (x + 255) & ~static_cast<size_t>(255); };
    const size_t slots = 2 * static_cast<size_t>(p.max_ctas) * p.rows_per;
    p.recs = kFarAt + up(sizeof(uint32_t) * static_cast<size_t>(a.R));
    p.ml = p.recs + up(sizeof(Rec) * p.max_ctas);
    p.part = p.ml + up(slots * sizeof(float2));
    p.total = p.part + up(slots * p.DVP * sizeof(float));
    return true;
}

template <int DP, int DVP, int NT, bool SPLIT, bool BESIDE = false>
cudaError_t launch(const Work& w, const CUtensorMap* maps, int rpb, cudaStream_t s) {
    using C = Cfg<DP, DVP, NT, SPLIT>;
    auto kernel = k_cache_attn_mma<DP, DVP, NT, SPLIT, BESIDE>;
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = uint64_t{1} << (dev & 63);
    if (!(done.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
        if (e != cudaSuccess) return e;
        done.fetch_or(bit, std::memory_order_relaxed);
    }
    if ((e = launch_early(dim3(w.ctas), dim3(kThreads), C::SMEM, s, kernel, maps[0], maps[1], w)) != cudaSuccess) return e;
    using E = typename std::conditional<SPLIT, float, __nv_bfloat16>::type;
    return launch_early(dim3(w.ctas, w.rows_per / rpb), dim3(256), 0, s, k_cache_join<DVP, E>, w, rpb, w.a.status);
}

}  // namespace

bool cache_attn_mma_supported(const CacheAttnArgs& a) {
    Plan p;
    return plan_of(a, p);
}

uint32_t* cache_attn_far(uint8_t* ws) { return reinterpret_cast<uint32_t*>(ws + kFarAt); }

size_t cache_attn_mma_workspace(const CacheAttnArgs& a) {
    Plan p;
    return plan_of(a, p) ? p.total : 256;
}

CacheBox cache_attn_mma_box(const CacheAttnArgs& a) {
    Plan p;
    plan_of(a, p);
    return {p.DP < 128 ? p.DP : 128, p.DVP < 128 ? p.DVP : 128, a.P < kTile ? a.P : kTile};
}

cudaError_t launch_cache_attn_mma(const CacheAttnArgs& a, const CUtensorMap* maps, uint8_t* ws, const uint32_t* far, cudaStream_t s) {
    Plan p;
    if (!plan_of(a, p)) return cudaErrorInvalidValue;
    Work w;
    w.a = a;
    w.rows_per = p.rows_per;
    w.far = far;
    // no more CTAs than the longest table rows have tiles
    const int64_t groups = (static_cast<int64_t>(a.max_q > 0 ? a.max_q : 1) * a.G + p.rows_per - 1) / p.rows_per;
    const double most = ((static_cast<int64_t>(a.max_pages) * a.P + kTile - 1) / kTile + kExtra) * static_cast<double>(a.Hkv) * a.R * groups;
    const int64_t ctas = static_cast<int64_t>(std::min(sm_count(), kMaxSms)) * p.occ;
    w.ctas = static_cast<int>(std::min(most, static_cast<double>(ctas)));
    w.recs = reinterpret_cast<Rec*>(ws + p.recs);
    w.ml = reinterpret_cast<float2*>(ws + p.ml);
    w.part = reinterpret_cast<float*>(ws + p.part);
    const uintptr_t qa = a.dtype == BPA_BF16 ? 7 : 15;
    w.vec_q = (reinterpret_cast<uintptr_t>(a.q) & qa) == 0 && a.qs[0] % 4 == 0 && a.qs[1] % 4 == 0;
    w.vec_o = a.dtype == BPA_BF16 && (reinterpret_cast<uintptr_t>(a.o) & 3) == 0 && a.os[0] % 2 == 0 && a.os[1] % 2 == 0;
    // Rows of a join block: few when an item is cut into many pieces, whose loads its warps then share.  Always
    // eight: three long requests 125.6 us against 123.5, one short one 12.3 against 11.9; always one: 62.7
    // against 45.1 (8 to 48 rows), 101.9 against 99.2 (64 requests of 4).
    const int64_t pieces = w.ctas / (static_cast<int64_t>(a.R) * a.Hkv);
    const int rpb = pieces <= 4 ? 8 : pieces <= 16 ? 4 : pieces <= 64 ? 2 : 1;
    const bool f32 = a.dtype == BPA_FP32;
    if (far) {                         // more than kFewRows rows (so NT is 2), bf16, head dims up to 128
        if (p.DP == 64) return launch<64, 64, 2, false, true>(w, maps, rpb, s);
        return p.DVP == 64 ? launch<128, 64, 2, false, true>(w, maps, rpb, s) : launch<128, 128, 2, false, true>(w, maps, rpb, s);
    }
#define BPA_CACHE_CASE(DP_, DVP_) \
    if (p.DP == DP_ && p.DVP == DVP_) \
        return p.NT == 1 ? f32 ? launch<DP_, DVP_, 1, true>(w, maps, rpb, s) : launch<DP_, DVP_, 1, false>(w, maps, rpb, s) \
                         : f32 ? launch<DP_, DVP_, 2, true>(w, maps, rpb, s) : launch<DP_, DVP_, 2, false>(w, maps, rpb, s);
    BPA_CACHE_CASE(64, 64)
    BPA_CACHE_CASE(128, 64)
    BPA_CACHE_CASE(128, 128)
    BPA_CACHE_CASE(256, 128)
    BPA_CACHE_CASE(256, 256)
#undef BPA_CACHE_CASE
    return cudaErrorInvalidValue;
}

}  // namespace bpa
