// Device helpers of the row operators (norm.hip, moe.hip): eight bf16 values a
// 16-byte piece, fp32 arithmetic, one rounding at the end.
#pragma once

#include "device_common.h"

namespace qg {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));

__device__ __forceinline__ void unpack8(u32x4 v, float* f) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        f[2 * j] = bf16_to_f32(w[j] & 0xffffu);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
    }
}

// eight fp32 values rounded to bf16 (nearest even)
__device__ __forceinline__ u32x4 pack8(const float* f) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        w[j] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{f[2 * j], f[2 * j + 1]}, bf16x2));
    return u32x4{w[0], w[1], w[2], w[3]};
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}

}  // namespace qg
