// 8-bit codes of rows and the reciprocal root of a norm (norm.hip, rope.hip).
#pragma once

#include "formats.h"
#include "rows.h"

namespace qg {

// Four quotients -> four codes.  |q| <= q_max up to roundings, which still round
// to the largest code: no clamp here.
template <class Fmt>
__device__ __forceinline__ uint32_t encode4(const float* q) {
    if constexpr (std::is_same<Fmt, FmtE4M3>::value) {
        int c = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
        return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], c, true);
    } else {
        // q + 1.5 2^23 has the half-even rounding of q in its lowest byte
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) c[j] = __float_as_uint(q[j] + 12582912.0f);
        return __builtin_amdgcn_perm(c[1], c[0], 0x0c0c0400u) | __builtin_amdgcn_perm(c[3], c[2], 0x04000c0cu);
    }
}

// The scale of a row and its codes: y times the rounded reciprocal of s (within
// one unit in the last place of the IEEE quotient y / s); a scale too small for
// a finite reciprocal divides.  The scale is the row's own maximum over q_max, so
// |y / s| exceeds q_max by roundings only -- except where s is subnormal, a whole
// number of steps of 2^-149 that max|y| / q_max may be far from (max|y| = 178
// steps: an int8 scale of one).  There the quotient is clamped.  EXACT: one correction of
// the product, with which the codes are those of the IEEE quotient (quant_act_per_token's)
// for every bf16 y that a row may hold, as an exhaustive check has shown, and for fp32 y
// but where the quotient's last bit decides a tie.
struct RowScale {
    float s, r;
    bool fast;
    template <class Fmt>
    __device__ static __forceinline__ RowScale of(float amax) {
        RowScale q;
        q.s = amax / Fmt::qmax;                              // IEEE fp32 quotient
        q.r = 1.0f / q.s;
        q.fast = q.s >= 0x1p-100f;
        return q;
    }
    template <class Fmt, bool EXACT = false>
    __device__ __forceinline__ uint2 codes(const float* y) const {
        if (s == 0.0f) return make_uint2(0u, 0u);
        float q[8];
        if (fast && (!EXACT || s < __builtin_inff())) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                q[j] = y[j] * r;
                if constexpr (EXACT) q[j] = fmaf(fmaf(-q[j], s, y[j]), r, q[j]);
            }
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                q[j] = y[j] / s;
                if (fabsf(q[j]) > Fmt::qmax) q[j] = copysignf(Fmt::qmax, q[j]);
            }
        }
        return make_uint2(encode4<Fmt>(q), encode4<Fmt>(q + 4));
    }
};

// 1 / sqrt(sum * inv_K + eps) in fp64 from the hardware's estimate and one Newton step,
// rounded once.
__device__ __forceinline__ float rstd_of(double sum, double inv_K, float eps) {
    const double v = fma(sum, inv_K, (double)eps);           // eps > 0
    const double r = __builtin_amdgcn_rsq(v);
    return (float)fma(r * 0.5, fma(-v * r, r, 1.0), r);
}

}  // namespace qg
