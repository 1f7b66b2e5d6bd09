// rope_api.cu - the C entry points of the norms of q and k with the position rotation (declared in
// include/bpa.h): argument checks, workspace and launches.
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <nvtx3/nvToolsExt.h>

#include "bpa.h"
#include "bpa_internal.h"
#include "rope.h"

using namespace bpa;

namespace {

constexpr size_t kHeader = 256;                  // the status word
constexpr int64_t kMost = int64_t{1} << 30;      // rows

bpa_status fail(bpa_status st, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof buf, fmt, ap);
    va_end(ap);
    set_last_error(buf);
    return st;
}

struct NvtxRange {
    explicit NvtxRange(const char* name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange&) = delete;
    NvtxRange& operator=(const NvtxRange&) = delete;
};

bpa_status cuda_status(cudaError_t e, const char* what) {
    return e == cudaSuccess ? BPA_OK : fail(BPA_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

// Sizes, strides and modes; pointers are not looked at.
bpa_status make_rope(const bpa_rope_desc* c, RopeArgs& a) {
    if (!c) return fail(BPA_ERR_INVALID_ARG, "descriptor is NULL");
    if (c->struct_size != sizeof(bpa_rope_desc))
        return fail(BPA_ERR_INVALID_ARG, "struct_size is %u, expected %zu", c->struct_size, sizeof(bpa_rope_desc));
    if (c->dtype != BPA_BF16 && c->dtype != BPA_FP32) return fail(BPA_ERR_INVALID_ARG, "unknown dtype %d", c->dtype);
    if (c->reserved) return fail(BPA_ERR_INVALID_ARG, "reserved must be 0");
    if (c->B < 1 || c->S < 0 || static_cast<int64_t>(c->B) * c->S > kMost)
        return fail(BPA_ERR_INVALID_ARG, "need B >= 1, S >= 0, B * S <= 2^30");
    if (c->Hq < 0 || c->Hkv < 0 || c->Hq + static_cast<int64_t>(c->Hkv) < 1)
        return fail(BPA_ERR_INVALID_ARG, "Hq and Hkv must be >= 0, one of them above");
    if (c->Hq > 65535 || c->Hkv > 65535) return fail(BPA_ERR_UNSUPPORTED, "more than 65535 heads");
    if (c->d < 1) return fail(BPA_ERR_INVALID_ARG, "d must be >= 1");
    if (c->d > 512) return fail(BPA_ERR_UNSUPPORTED, "head dim %d: at most 512", c->d);
    if (c->rot < 0 || c->rot > c->d || c->rot % 2)
        return fail(BPA_ERR_INVALID_ARG, "rot (%d) must be even and in [0, d]", c->rot);
    if (c->norm && !(c->eps >= 1.17549435e-38f && c->eps <= 3.402823466e38f))
        return fail(BPA_ERR_INVALID_ARG, "eps must be a positive normal number");
    if (!c->norm && (c->q_weight || c->k_weight)) return fail(BPA_ERR_INVALID_ARG, "weights without a norm");
    if (c->rot && !c->inv_freq) return fail(BPA_ERR_INVALID_ARG, "inv_freq is NULL");
    memset(&a, 0, sizeof a);
    a.dtype = c->dtype;
    a.B = c->B;
    a.S = c->S;
    a.d = c->d;
    a.rot = c->rot;
    a.interleaved = c->interleaved != 0;
    a.norm = c->norm != 0;
    a.eps = c->eps;
    a.far = c->norm ? -ilogbf(sqrtf(c->eps)) : 0;
    a.pos = c->positions;
    a.freq = c->inv_freq;
    const int64_t* in[2] = {c->q_strides, c->k_strides};
    const int64_t* out[2] = {c->qo_strides, c->ko_strides};
    for (int i = 0; i < 2; ++i) {
        RopeSide& t = a.side[i];
        t.H = i ? c->Hkv : c->Hq;
        t.x = i ? c->k : c->q;
        t.w = i ? c->k_weight : c->q_weight;
        for (int j = 0; j < 3; ++j) {
            t.xs[j] = in[i][j];
            t.ys[j] = out[i][j];
            if (t.H && (t.xs[j] < 0 || t.ys[j] < 0)) return fail(BPA_ERR_INVALID_ARG, "strides must be >= 0");
        }
    }
    return BPA_OK;
}

// A tensor that is written: no two of its rows or heads may lie over one another for a stride of 0.
bool written_ok(const RopeArgs& a, const RopeSide& t, const int64_t st[3]) {
    return (a.B == 1 || st[0]) && (a.S <= 1 || st[1]) && (t.H <= 1 || st[2]);
}

bool empty(const RopeArgs& a) { return a.S == 0; }

size_t workspace_of(const RopeArgs& a) { return kHeader + sizeof(float) * 2 * kRopeMaxBlocks * static_cast<size_t>((a.d + 31) / 32 * 32); }

}  // namespace

extern "C" {

bpa_status bpa_rope_fwd(const bpa_rope_desc* desc, void* q_out, void* k_out, void* stream) {
    const NvtxRange range("bpa_rope_fwd");
    RopeArgs a;
    const bpa_status st = make_rope(desc, a);
    if (st != BPA_OK) return st;
    a.side[0].y = q_out;
    a.side[1].y = k_out;
    for (const RopeSide& t : a.side) {
        if (t.H == 0) continue;
        if (!written_ok(a, t, t.ys)) return fail(BPA_ERR_INVALID_ARG, "an output's strides must be above 0");
        if (!empty(a) && (!t.x || !t.y)) return fail(BPA_ERR_INVALID_ARG, "q, k, q_out or k_out is NULL");
    }
    if (empty(a)) return BPA_OK;
    return cuda_status(launch_rope_fwd(a, static_cast<cudaStream_t>(stream)), "norm and rotation launch");
}

size_t bpa_rope_workspace_size(const bpa_rope_desc* desc) {
    RopeArgs a;
    return make_rope(desc, a) == BPA_OK ? workspace_of(a) : 0;
}

bpa_status bpa_rope_bwd(const bpa_rope_desc* desc, const void* dq_out, const void* dk_out, void* dq, void* dk, float* dq_weight,
                        float* dk_weight, void* workspace, size_t workspace_bytes, void* stream) {
    const NvtxRange range("bpa_rope_bwd");
    RopeArgs a;
    const bpa_status st = make_rope(desc, a);
    if (st != BPA_OK) return st;
    if (!a.norm && (dq_weight || dk_weight)) return fail(BPA_ERR_INVALID_ARG, "gradients of weights without a norm");
    const void* grads[2] = {dq_out, dk_out};
    void* outs[2] = {dq, dk};
    float* dw[2] = {dq_weight, dk_weight};
    for (int i = 0; i < 2; ++i) {
        RopeSide& t = a.side[i];
        t.dy = grads[i];
        t.y = outs[i];
        t.dw = dw[i];
        if (t.H == 0) continue;
        if (!written_ok(a, t, t.xs)) return fail(BPA_ERR_INVALID_ARG, "a gradient's strides must be above 0");
        if (!empty(a) && ((a.norm && !t.x) || !t.y || !t.dy))
            return fail(BPA_ERR_INVALID_ARG, "q, k, dq_out, dk_out, dq or dk is NULL");
        if (!a.norm) t.x = t.y;        // not read, and may be NULL: copies of no bytes still want an address
    }
    if (!workspace) return fail(BPA_ERR_WORKSPACE, "workspace is NULL (need %zu bytes)", workspace_of(a));
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return fail(BPA_ERR_WORKSPACE, "workspace must be 256-byte aligned");
    if (workspace_bytes < workspace_of(a))
        return fail(BPA_ERR_WORKSPACE, "workspace has %zu bytes, needs %zu", workspace_bytes, workspace_of(a));
    a.status = static_cast<uint32_t*>(workspace);
    a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + kHeader);
    return cuda_status(launch_rope_bwd(a, static_cast<cudaStream_t>(stream)), "norm and rotation launch");
}

}  // extern "C"
