// What happens to a product's fp32 results before they are stored: nothing but
// the rounding (NoEpilogue), or act(v + bias[n]) + residual[m, n] first.  A
// kernel fetches the bias and residual of the results that a thread stores
// together (an In) while other work is under way, and applies them before the
// first store: y may be the residual's memory, so the compiler may not move a
// load over such a store.  Loaded bits stay as they are until then: a conversion
// next to the load would wait for it.  Whether there is a residual and an
// activation is part of the type: fetched residuals cost the products of few rows
// up to 19 registers, and the branch over the activations' code some time per
// tile, which the wide layers that have neither do not pay.  A bias alone, 1 / 8 /
// 16 x 4096 x 28672 (plain product 13.0 / 13.8 / 14.5 us), costs 0.2 / 0.1 / 0.1 us
// so, 0.8 / 0.6 / 0.6 with the activation decided at run time and 1.2 / 0.7 / 0.9
// with the residual too.  Beside a residual the activation stays a branch: a form
// without it would be one more copy of every kernel for 1 to 2 % either way (us with
// the branch and without: 16 x 14336 x 4096 13.7 and 13.8, 8 x 14336 x 4096 11.8 and 11.7,
// 16 x 28672 x 8192 36.6 and 37.0, 16 x 4096 x 28672 15.7 and 15.6).
#pragma once

#include "device_common.h"

namespace qg {

struct NoEpilogue {
    using out_ptr = uint16_t* __restrict__;
    static constexpr bool kActive = false;
    template <int C>
    struct In {};
    __device__ __forceinline__ uint32_t bias_bits(int) const { return 0u; }
    // residuals (and with BIAS also biases) of the results i < C at row(i), col(i); results
    // outside M x N get the nearest one's, which saves a branch each
    template <bool BIAS, int C, class Row, class Col>
    __device__ __forceinline__ void fetch(In<C>&, int, int, Row, Col) const {}
    template <int C, class V>
    __device__ __forceinline__ void apply(V&, const In<C>&) const {}
    template <int C, class V>
    __device__ __forceinline__ void apply(V&, const In<C>&, uint32_t) const {}
};

// qg_activation of include/qgemm.h
enum { ACT_NONE = 0, ACT_RELU = 1, ACT_GELU = 2, ACT_GELU_TANH = 3, ACT_SILU = 4 };

// The activations run once per output on accumulators that are about to be
// rounded to 8 bits of mantissa: hardware exp2 and reciprocal (1 unit in the
// last place each; the exponent's own rounding adds |z| 2^-24).

// x sigmoid(z); far below zero the denominator is infinite and the result -0
__device__ __forceinline__ float x_sigmoid(float x, float z) {
    return x * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * z));
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
    // past |x| = 2^63 the square would overflow: the tail is zero from 20 on, where
    // b also keeps +inf from meeting it (-inf times zero stays NaN)
    const float b = fminf(a, 20.0f);
    const float tail = p * t * __builtin_amdgcn_exp2f(-0.721347520f * b * b);
    return x < 0.0f ? x * tail : fmaf(-b, tail, x);
}

template <int C, class V>
__device__ __forceinline__ void activate(V& v, int act) {
    switch (act) {                               // uniform: one branch for all C values
        case ACT_RELU:
            // the maximum that keeps NaN: sums that overflowed with both signs stay visible
#pragma unroll
            for (int i = 0; i < C; ++i) v[i] = __builtin_elementwise_maximum(v[i], 0.0f);
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

template <bool RES, bool ACT>
struct Epilogue {
    using out_ptr = uint16_t*;
    static constexpr bool kActive = true;
    static constexpr bool kResidual = RES, kActivation = ACT;
    const uint16_t* bias;                        // [N] or null
    const uint16_t* residual;                    // [M, N], read if RES
    int act;                                     // qg_activation, looked at if ACT

    template <int C>
    struct In {
        uint32_t b[C], r[C];                     // bf16 bits
    };
    // the bits as loaded: nothing waits for them before they are used
    __device__ __forceinline__ uint32_t bias_bits(int n) const { return bias ? bias[n] : 0u; }
    // eight consecutive biases (n % 2 == 0; the pointer is 4-byte aligned)
    __device__ __forceinline__ void bias8(float* b, int n) const {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t w = bias ? reinterpret_cast<const uint32_t*>(bias + n)[j] : 0u;
            b[2 * j] = bf16_to_f32(w & 0xffffu);
            b[2 * j + 1] = __uint_as_float(w & 0xffff0000u);
        }
    }
    template <bool BIAS, int C, class Row, class Col>
    __device__ __forceinline__ void fetch(In<C>& in, int M, int N, Row row, Col col) const {
        if (RES) {
#pragma unroll
            for (int i = 0; i < C; ++i) in.r[i] = residual[(size_t)min(row(i), M - 1) * N + min(col(i), N - 1)];
        }
        if (BIAS && bias) {
#pragma unroll
            for (int i = 0; i < C; ++i) in.b[i] = bias[min(col(i), N - 1)];
        }
    }
    template <int C, class V>
    __device__ __forceinline__ void apply(V& v, const In<C>& in) const {
        if (bias) {
#pragma unroll
            for (int i = 0; i < C; ++i) v[i] += bf16_to_f32(in.b[i]);
        }
        finish<C>(v, in);
    }
    // results of one column, its bias bits already there
    template <int C, class V>
    __device__ __forceinline__ void apply(V& v, const In<C>& in, uint32_t bits) const {
        const float b = bf16_to_f32(bits);
#pragma unroll
        for (int i = 0; i < C; ++i) v[i] += b;
        finish<C>(v, in);
    }

private:
    template <int C, class V>
    __device__ __forceinline__ void finish(V& v, const In<C>& in) const {
        if (ACT) activate<C>(v, act);
        if (RES) {
#pragma unroll
            for (int i = 0; i < C; ++i) v[i] += bf16_to_f32(in.r[i]);
        }
    }
};

}  // namespace qg
