// Arithmetic on rows shared by the norms: bf16 and e4m3 conversions, a maximum
// that keeps NaN, and sums over a warp.
#pragma once
#include <cuda_bf16.h>

#include "a2av_internal.cuh"

namespace a2av {

constexpr float kLow8 = 448.0f;     // largest finite e4m3
constexpr float kZeroRow = 1e-30f;  // an 8-bit row whose maximum is below this is stored as zeros

// NaN-keeping maximum: a NaN anywhere in a row has to reach its scale.
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// Rounded to nearest even, values past 448 (one rounding of 448/a away at most) to 448.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t d;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
    return d;
}

__device__ __forceinline__ float lo_f(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ float hi_f(uint32_t v) { return __uint_as_float(v & 0xffff0000u); }

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

}  // namespace a2av
