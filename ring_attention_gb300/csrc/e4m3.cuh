// e4m3.cuh - conversions of the 8-bit cache's codes.
#pragma once

#include <cuda_fp8.h>

#include "common.cuh"

namespace bpa {

// round to nearest even; |x| <= 448 here, NaN gives NaN, infinities 448
BPA_DEV uint32_t e4m3_pair(float lo, float hi) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}
BPA_DEV float from_e4m3(uint8_t c) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(c, __NV_E4M3)));
}
// four codes at another scale: e4m3(code * ratio)
BPA_DEV uint32_t rescaled4(uint32_t y, float ratio) {
    return e4m3_pair(from_e4m3(y & 0xff) * ratio, from_e4m3((y >> 8) & 0xff) * ratio) |
           e4m3_pair(from_e4m3((y >> 16) & 0xff) * ratio, from_e4m3(y >> 24) * ratio) << 16;
}

}  // namespace bpa
