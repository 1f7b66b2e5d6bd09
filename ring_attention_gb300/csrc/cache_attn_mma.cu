// cache_attn_mma.cu - choice of tiles, workspace and launch of the few-row cache attention.
#include "cache_attn_mma.cuh"

namespace bpa {

using namespace cache_mma;

namespace {

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

cudaError_t launch_cache_attn_mma(const CacheAttnArgs& a, const CUtensorMap* maps, uint8_t* ws, const uint32_t* far, const Pieces* more,
                                  cudaStream_t s) {
    Plan p;
    if (!plan_of(a, p)) return cudaErrorInvalidValue;
    Work w = {};
    w.a = a;
    if (more) w.more = *more;
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
    return a.tree ? launch_trees(w, p.DP, p.DVP, p.NT, maps, rpb, s) : launch_any<false>(w, p.DP, p.DVP, p.NT, maps, rpb, s);
}

}  // namespace bpa
