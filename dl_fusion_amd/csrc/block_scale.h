// Block scales of e4m3 codes on the device: a block's largest magnitude, its scale and its codes.
#pragma once

#include "device_common.h"

namespace dlf {

constexpr int kScaleBlock = 128;            // columns that share a scale
constexpr float kLeastMax = 0x1p-110f;      // a block's largest magnitude is taken as at least this:
                                            // 448 / amax stays finite and amax / 448 normal
// |v|, 0 for what is not finite
__device__ __forceinline__ float finite_abs(float v) {
    const float a = fabsf(v);
    return a < INFINITY ? a : 0.0f;
}

// Four codes of fp32(v * inv), packed little-endian: saturated at +-448; NaN passes the comparison and
// the conversion encodes it.
__device__ __forceinline__ uint32_t e4m3_x4(const float* v, float inv) {
    float p[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        p[i] = __fmul_rn(v[i], inv);
        p[i] = fabsf(p[i]) > 448.0f ? copysignf(448.0f, p[i]) : p[i];
    }
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(p[0], p[1], 0, false);
    w = __builtin_amdgcn_cvt_pk_fp8_f32(p[2], p[3], w, true);
    return static_cast<uint32_t>(w);
}

}  // namespace dlf
