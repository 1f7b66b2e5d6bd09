// cache_pieces.h - what the cache attention's CTAs leave for the join of items that they cut.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace bpa {
namespace cache_mma {

// The workspace, and the join's list of pieces in shared memory, are sized for these: SMs, CTAs of an SM of the few-row
// kernel, CTAs of the tensor-core kernel under trees.
constexpr int kMaxSms = 160, kMaxOcc = 4, kMaxTcCtas = kMaxSms;
constexpr int kMaxPieces = kMaxSms * kMaxOcc + kMaxTcCtas;

struct Rec {                          // what a CTA leaves for the join
    int trail;                        // slot 1 holds the first of `trail` pieces of an item (0: none)
    int row0, hk, i0, nrows;          // that item
    uint32_t flags, where;            // this CTA's status
    int r;                            // the item's request
};
static_assert(sizeof(Rec) == 32, "record");

// Pieces that another kernel has left for the same join.
struct Pieces {
    Rec* recs;                        // [ctas]
    float2* ml;                       // [2 ctas][rows_per]
    float* part;                      // [2 ctas][DVP / 4][rows_per][4]
    int ctas, rows_per;
};

}  // namespace cache_mma
}  // namespace bpa
