// cache_keep.cu - the accepted tokens of a step moved to the end of the context, in the 8-bit cache.
//
// Token keep[i] of the step goes to place ctx + i.  A page's scale becomes the largest of what it then holds (its
// own, if tokens in front of the moved ones stay in it; those of the pages that its tokens come from), and
// what comes with a smaller one is rounded again: code' = e4m3(code * (old / new)), which powers of two make
// exact but below e4m3's smallest normal number.
//
// A warp per request, head and tensor, pages and tokens in ascending order.  A token never moves up
// (keep[i] >= i), so a place that is written has been read, whether its token went elsewhere or stays: the
// sources of later tokens lie behind it, and the pages that they come from keep their scales until then.
// Bounded by the latency of a warp's chain (lengths, path, page ids, scales, codes, page after page): 4 requests of 8
// heads 7.4 us with the status word's clearing (1.5), 256 requests with paths of up to 30 tokens over pages of 16
// 12.6 us, in which it moves 6 MB.
#include "cache.h"
#include "common.cuh"
#include "e4m3.cuh"

namespace bpa {
namespace {

constexpr int kWarps = 4;

template <bool WIDE>
__global__ void __launch_bounds__(32 * kWarps) k_cache_keep(const KeepArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t item = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    wait_for_previous();
    const int r = static_cast<int>(item / (2 * a.Hkv)), hw = static_cast<int>(item - static_cast<int64_t>(r) * 2 * a.Hkv);
    if (r >= a.R) return;
    const int h = hw >> 1;
    const bool is_v = hw & 1;
    const int cnt = a.count[r];
    if (cnt == 0) return;
    const int row0 = a.cu_q[r], n = a.cu_q[r + 1] - row0, len = a.kv_lens[r], ctx = len - n;
    const int32_t *keep = a.keep + static_cast<int64_t>(r) * a.max_keep, *table = a.table + static_cast<int64_t>(r) * a.max_pages;
    // the whole request is looked over before anything moves, by each of its warps alike
    bool ok = row0 >= 0 && n >= 0 && row0 <= a.T - n && ctx >= 0 && len <= static_cast<int64_t>(a.max_pages) * a.P && cnt > 0 &&
              cnt <= n && cnt <= a.max_keep;
    if (ok) {
        bool fine = true;
        for (int i = lane; i < cnt; i += 32) {
            const int x = keep[i];
            if (x < 0 || x >= n || (i && x <= keep[i - 1])) {
                fine = false;
                continue;
            }
            const int from = table[(ctx + x) / a.P], to = table[(ctx + i) / a.P];
            fine = fine && from >= 0 && from < a.num_pages && to >= 0 && to < a.num_pages;
        }
        ok = __all_sync(0xffffffffu, fine);
    }
    if (!ok) {
        if (hw == 0 && lane == 0) report(a.status, ST_CHECK, 0xCD8);
        return;
    }
    const int c = is_v ? a.dv : a.d;
    float* scales = (is_v ? a.vscale : a.kscale) + h;
    uint8_t* codes = (is_v ? a.vc + h * a.vcs[1] : a.kc + h * a.kcs[1]);
    const int64_t ps = is_v ? a.vcs[0] : a.kcs[0], ts = is_v ? a.vcs[2] : a.kcs[2];
    const int units = WIDE ? c / 16 : 1, down = 32 / units, li = WIDE ? lane / units : 0, lu = WIDE ? lane % units : lane;
    auto scale_of = [&](int id) { return scales + static_cast<int64_t>(id) * a.Hkv; };
    // rows [0, m) at `to` (a row every ts): row i is that at from(i) times ratio(i)
    auto move = [&](int m, auto from, auto ratio, uint8_t* to) {
        if (WIDE) {
            for (int b = 0; b < m; b += 2 * down) {
                uint4 x[2];
                float f[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int i = b + k * down + li;
                    if (li < down && i < m) {
                        x[k] = *reinterpret_cast<const uint4*>(from(i) + 16 * lu);
                        f[k] = ratio(i);
                    }
                }
                __syncwarp();          // read before any of them is written
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int i = b + k * down + li;
                    if (li >= down || i >= m) continue;
                    if (f[k] != 1.f)
                        x[k] = make_uint4(rescaled4(x[k].x, f[k]), rescaled4(x[k].y, f[k]), rescaled4(x[k].z, f[k]), rescaled4(x[k].w, f[k]));
                    *reinterpret_cast<uint4*>(to + i * ts + 16 * lu) = x[k];
                }
                __syncwarp();
            }
        } else {
            for (int i = 0; i < m; ++i) {
                const uint8_t* p = from(i);
                const float f = ratio(i);
                for (int e = lu; e < c; e += 32) {         // a lane's own channels: read, then written
                    const uint8_t y = p[e];
                    to[i * ts + e] = f == 1.f ? y : static_cast<uint8_t>(e4m3_pair(from_e4m3(y) * f, 0.f));
                }
                __syncwarp();
            }
        }
    };
    for (int j = ctx / a.P; j * static_cast<int64_t>(a.P) < ctx + cnt; ++j) {
        const int begin = j * a.P, front = max(ctx - begin, 0);          // tokens of this page in front of the step's
        const int i0 = max(begin - ctx, 0), i1 = static_cast<int>(min(static_cast<int64_t>(cnt), static_cast<int64_t>(begin) + a.P - ctx));
        const int page = table[j];
        const float old = *scale_of(page);
        float top = front ? old : 0.f;
        bool moves = false;
        for (int i = i0 + lane; i < i1; i += 32) {
            top = fmaxf(top, *scale_of(table[(ctx + keep[i]) / a.P]));
            moves |= keep[i] != i;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (!__any_sync(0xffffffffu, moves) && top == old) continue;      // everything is where it belongs
        uint8_t* base = codes + page * ps;
        const float grown = top > 0.f ? old / top : 1.f;
        if (front && grown != 1.f)
            move(front, [&](int i) { return base + i * ts; }, [&](int) { return grown; }, base);
        move(i1 - i0,
             [&](int i) {
                 const int at = ctx + keep[i0 + i];
                 return codes + table[at / a.P] * ps + (at % a.P) * ts;
             },
             [&](int i) { return top > 0.f ? *scale_of(table[(ctx + keep[i0 + i]) / a.P]) / top : 1.f; },
             base + static_cast<int64_t>(ctx + i0 - begin) * ts);
        __syncwarp();
        if (lane == 0) *scale_of(page) = top;
        __syncwarp();
    }
}

}  // namespace

cudaError_t launch_cache_keep(const KeepArgs& a, cudaStream_t s) {
    // rows in units of 16 bytes where everything is aligned to them
    uintptr_t all = reinterpret_cast<uintptr_t>(a.kc) | reinterpret_cast<uintptr_t>(a.vc) | a.d | a.dv;
    for (int i = 0; i < 3; ++i) all |= static_cast<uintptr_t>(a.kcs[i]) | static_cast<uintptr_t>(a.vcs[i]);
    const int64_t items = static_cast<int64_t>(a.R) * 2 * a.Hkv;
    const dim3 grid(static_cast<unsigned>((items + kWarps - 1) / kWarps));
    return launch_early(grid, dim3(32 * kWarps), 0, s, all % 16 == 0 ? k_cache_keep<true> : k_cache_keep<false>, a);
}

}  // namespace bpa
