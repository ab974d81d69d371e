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

// ---- streamed rows -----------------------------------------------------------
// Bytes that nothing reads again soon (an input at its last use, an output that
// the caches cannot hold until its reader comes) go past the caches with the
// non-temporal hint, which leaves them to what is read again.
template <bool STREAM, class T>
__device__ __forceinline__ T load_row(const T* p) {
    if constexpr (STREAM) return __builtin_nontemporal_load(p);
    else return *p;
}
template <bool STREAM, class T>
__device__ __forceinline__ void store_row(T* p, T v) {
    if constexpr (STREAM) __builtin_nontemporal_store(v, p);
    else *p = v;
}
// rows that count as such: more than the XCDs' L2s hold together
constexpr size_t kStreamBytes = size_t(32) << 20;

// ---- wave reductions on DPP moves ------------------------------------------
// Row shifts by 1, 2, 4, 8 and the row broadcasts 15 and 31 leave the result of
// all 64 lanes in lane 63, a few cycles a step (a shuffle through LDS takes
// about a hundred).  Lanes without a source keep `none`, the identity.
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ uint32_t dpp_u32(uint32_t none, uint32_t v) {
    return (uint32_t)__builtin_amdgcn_update_dpp((int)none, (int)v, CTRL, ROWS, 0xf, false);
}
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ float dpp(float v) {
    return __uint_as_float(dpp_u32<CTRL, ROWS>(0u, __float_as_uint(v)));
}
template <int CTRL, int ROWS = 0xf>
__device__ __forceinline__ double dpp(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint64_t lo = dpp_u32<CTRL, ROWS>(0u, (uint32_t)u);
    const uint64_t hi = dpp_u32<CTRL, ROWS>(0u, (uint32_t)(u >> 32));
    return __builtin_bit_cast(double, lo | (hi << 32));
}
__device__ __forceinline__ float lane63(float v) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_readlane(__float_as_int(v), 63));
}
__device__ __forceinline__ double lane63(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint64_t lo = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)u, 63);
    const uint64_t hi = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(u >> 32), 63);
    return __builtin_bit_cast(double, lo | (hi << 32));
}

// The sum over the wave's lanes (float or double), in every lane.
template <class T>
__device__ __forceinline__ T wave_sum(T v) {
    v += dpp<0x111>(v);
    v += dpp<0x112>(v);
    v += dpp<0x114>(v);
    v += dpp<0x118>(v);
    v += dpp<0x142, 0xa>(v);
    v += dpp<0x143, 0xc>(v);
    return lane63(v);
}
// The largest magnitude; a NaN counts as larger than any number and stays one.
__device__ __forceinline__ float max_abs(float a, float b) { return __builtin_elementwise_maximum(a, fabsf(b)); }
// Over the wave's lanes, for a >= 0 or NaN: their bits order as the values do.
__device__ __forceinline__ float wave_max_abs(float a) {
    uint32_t u = __float_as_uint(a) & 0x7fffffffu;
    u = max(u, dpp_u32<0x111>(0u, u));
    u = max(u, dpp_u32<0x112>(0u, u));
    u = max(u, dpp_u32<0x114>(0u, u));
    u = max(u, dpp_u32<0x118>(0u, u));
    u = max(u, dpp_u32<0x142, 0xa>(0u, u));
    u = max(u, dpp_u32<0x143, 0xc>(0u, u));
    return lane63(__uint_as_float(u));
}

}  // namespace qg
