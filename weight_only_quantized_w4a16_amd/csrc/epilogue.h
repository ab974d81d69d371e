// What happens to a product's fp32 results before they are stored: nothing but
// the rounding (NoEpilogue), or act(v + bias[n]) + residual[m, n] first.  A
// kernel hands over the C results that a thread stores together, so that their
// residuals are all requested before the first store (y may be the residual's
// memory, and the compiler may not move a load over such a store).
#pragma once

#include "device_common.h"

namespace qg {

struct NoEpilogue {
    using out_ptr = uint16_t* __restrict__;
    // v[i] becomes the value of row row(i), column col(i); only those with live(i) are read
    template <int C, class V, class Live, class Row, class Col>
    __device__ __forceinline__ void apply(V&, int, Live, Row, Col) const {}
};

// qg_activation of include/qgemm.h
enum { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

// The activations run once per output on accumulators that are about to be
// rounded to 8 bits of mantissa: hardware exp2 and reciprocal (1 unit in the
// last place each; the exponent's own rounding adds |z| 2^-24).

// x sigmoid(z) without overflow: exp(-|z|) <= 1
__device__ __forceinline__ float x_sigmoid(float x, float z) {
    const float e = __builtin_amdgcn_exp2f(-1.44269504f * fabsf(z));
    return (z < 0.0f ? x * e : x) * __builtin_amdgcn_rcpf(1.0f + e);
}

// x Phi(x): the tail Phi(-|x|) = exp(-x^2 / 2) t P(t), t = 1 / (1 + 0.4 |x| /
// sqrt 2), with P the polynomial of degree 8 fitted to erfc(z) exp(z^2) / 2 over
// z >= 0 for the least relative error (1.3e-7), so small outputs keep their
// precision.
__device__ __forceinline__ float x_phi(float x) {
    const float a = fabsf(x);
    const float t = __builtin_amdgcn_rcpf(fmaf(0.282842712f, a, 1.0f));
    float p = 0.0251365686f;
    p = fmaf(p, t, -0.0914729705f);
    p = fmaf(p, t, 0.0845794443f);
    p = fmaf(p, t, -0.00283569511f);
    p = fmaf(p, t, 0.0707313687f);
    p = fmaf(p, t, 0.0842666882f);
    p = fmaf(p, t, 0.103921967f);
    p = fmaf(p, t, 0.11283476f);
    p = fmaf(p, t, 0.112837932f);
    // past |x| = 2^63 the square would overflow: the tail is zero long before
    const float b = fminf(a, 20.0f);
    const float tail = p * t * __builtin_amdgcn_exp2f(-0.721347520f * b * b);
    return x < 0.0f ? x * tail : fmaf(-x, tail, x);
}

template <int C, class V>
__device__ __forceinline__ void activate(V& v, int act) {
    switch (act) {                               // uniform: one branch for all C values
        case ACT_RELU:
#pragma unroll
            for (int i = 0; i < C; ++i) v[i] = fmaxf(v[i], 0.0f);
            break;
        case ACT_GELU:
#pragma unroll
            for (int i = 0; i < C; ++i) v[i] = x_phi(v[i]);
            break;
        case ACT_GELU_TANH:
            // 0.5 x (1 + tanh u) = x sigmoid(2 u), u = sqrt(2 / pi) (x + 0.044715 x^3)
#pragma unroll
            for (int i = 0; i < C; ++i) v[i] = x_sigmoid(v[i], v[i] * fmaf(0.0713548163f, v[i] * v[i], 1.59576912f));
            break;
        case ACT_SILU:
#pragma unroll
            for (int i = 0; i < C; ++i) v[i] = x_sigmoid(v[i], v[i]);
            break;
        default: break;
    }
}

struct Epilogue {
    using out_ptr = uint16_t*;
    const uint16_t* bias;                        // [N] or null
    const uint16_t* residual;                    // [M, N] or null
    int act;

    template <int C, class V, class Live, class Row, class Col>
    __device__ __forceinline__ void apply(V& v, int N, Live live, Row row, Col col) const {
        float r[C];
#pragma unroll
        for (int i = 0; i < C; ++i)
            r[i] = residual && live(i) ? bf16_to_f32(residual[(size_t)row(i) * N + col(i)]) : 0.0f;
        if (bias) {
#pragma unroll
            for (int i = 0; i < C; ++i) v[i] += live(i) ? bf16_to_f32(bias[col(i)]) : 0.0f;
        }
        activate<C>(v, act);
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] += r[i];
    }
};

}  // namespace qg
