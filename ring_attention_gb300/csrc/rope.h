// rope.h - norms of q and k with the position rotation: validated calls and kernel launchers of libbpa.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "bpa.h"

namespace bpa {

// One of the two tensors of a call.  Strides (b, s, h) in elements, the last dim contiguous.
struct RopeSide {
    int H;                             // heads; 0: none
    const void* x;                     // before norm and rotation
    int64_t xs[3];
    void* y;                           // forward: behind both (strides ys); backward: the gradient of x (strides xs)
    const void* dy;                    // backward: the gradient of what the forward pass wrote (strides ys)
    int64_t ys[3];
    const float* w;                    // [d] weights of the norm or null (ones)
    float* dw;                         // backward: [d] gradient of w or null
};

struct RopeArgs {
    int dtype, B, S, d, rot, interleaved, norm;
    float eps;
    int far;                           // sqrt(eps) times two to this lies in [1, 2)
    const int32_t* pos;                // [B, S] or null: the place in the sequence
    const float* freq;                 // [rot / 2] radians per position
    RopeSide side[2];                  // q, k
    float* part;                       // backward: [blocks][2][d] partial sums of the weights' gradients
    uint32_t* status;                  // backward: the workspace's status word
};

constexpr int kRopeMaxBlocks = 640;    // blocks of a call at most (four on each of 160 SMs)

cudaError_t launch_rope_fwd(const RopeArgs& a, cudaStream_t s);
cudaError_t launch_rope_bwd(const RopeArgs& a, cudaStream_t s);

}  // namespace bpa
