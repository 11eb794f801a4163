// kvd_q8.cuh -- e4m3 codes and their blocks' scales, shared by what writes, reads and
// attends pages of 8 bits.
#pragma once

#include <cuda_fp8.h>

#include "kvd_internal.cuh"

namespace kvd {

constexpr float kScaleLow = 5.421010862427522e-20f;   // 2^-64
constexpr float kScaleHigh = 1.8446744073709552e19f;  // 2^64

__device__ __forceinline__ bool scale_ok(float s) { return s >= kScaleLow && s <= kScaleHigh; }
// What a reader takes for a block's scale: 1 for one that cannot be.
__device__ __forceinline__ float scale_of(float s, uint32_t *err) {
    if (scale_ok(s)) return s;
    set_error(err, kErrBounds);
    return 1.0f;
}

// Four values to codes, to nearest even, 448 at most; four codes to values.
__device__ __forceinline__ uint32_t codes4(const float *x) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(x[0], x[1]), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(x[2], x[3]), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}
__device__ __forceinline__ void values4(uint32_t w, float *x) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w >> (16 * i)), __NV_E4M3);
        const float2 f = __half22float2(__half2(h));
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

}  // namespace kvd
