// The activation steps between two quantized products of a decoder block, each
// in one pass: the residual's addition with the root-mean-square norm, and the
// gated unit of the feed-forward layer, both with a bf16 output or with the
// per-token 8-bit codes and scales that the W8A8 and W4A8 products read.
//
//   rms_norm   h = x + residual, y = (h * rsqrt(mean(h^2) + eps)) * weight
//   swiglu     y = gate / (1 + exp(-gate)) * up
//   codes      s = max|y| / q_max (IEEE), q = rnd(y / s); a zero row: s = 0, q = 0;
//              a row with a NaN: s is NaN; with an infinity: infinite or NaN
//
// Everything between the bf16 inputs and the output is fp32 (the sum of squares
// fp64): y is rounded once, to bf16 or to its code, and h (stored as bf16)
// enters the norm unrounded.
// Both are bound by memory: a row is read once and stays in registers between
// the reductions and the encoding.  Graph-timed, on buffers in turn that no cache
// holds (as every figure of this file): norm with residual at 8191 x 8192 to bf16 /
// e4m3 90 / 79 us (5.9 TB/s; a copy 5.3), at 1 x 4096 2.6 / 2.9 us; swiglu at 8192 x
// 14336 116 / 103 us (6.1 / 5.7 TB/s), at 16 x 14336 2.3 / 3.9 us (an empty launch
// takes about 2).

#include <algorithm>

#include "codes.h"
#include "device_common.h"
#include "formats.h"
#include "launch.h"
#include "rows.h"

namespace qg {

struct FmtNone {                               // bf16 output only
    static constexpr float qmax = 1.0f;
};
template <class Fmt>
constexpr bool kCodes = !std::is_same<Fmt, FmtNone>::value;

// Reductions over the NT threads of a row, in a fixed order; every thread gets
// the result.  NT < 64: lanes of one wave, by shuffles; 64: a wave; more: one LDS
// word per wave (`red`, used once per launch) and a barrier.
template <int NT>
__device__ __forceinline__ double lanes_sum(double v) {
    if constexpr (NT >= 64) return wave_sum(v);
#pragma unroll
    for (int o = NT / 2; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
    return v;
}
template <int NT>
__device__ __forceinline__ float lanes_max(float v) {
    if constexpr (NT >= 64) return wave_max_abs(v);
#pragma unroll
    for (int o = NT / 2; o > 0; o >>= 1) v = max_abs(v, __shfl_xor(v, o, 64));
    return v;
}
template <int NT>
__device__ __forceinline__ double row_sum(double v, double* red) {
    v = lanes_sum<NT>(v);
    if constexpr (NT > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0;
#pragma unroll
        for (int w = 0; w < NT / 64; ++w) v += red[w];
    }
    return v;
}
template <int NT>
__device__ __forceinline__ float row_max(float v, float* red) {
    v = lanes_max<NT>(v);
    if constexpr (NT > 64) {
        if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < NT / 64; ++w) v = max_abs(v, red[w]);
    }
    return v;
}
// both at once: one barrier
template <int NT>
__device__ __forceinline__ void row_sum_max(double& sum, float& top, double* red_sum, float* red_max) {
    sum = lanes_sum<NT>(sum);
    top = lanes_max<NT>(top);
    if constexpr (NT > 64) {
        if ((threadIdx.x & 63) == 0) {
            red_sum[threadIdx.x >> 6] = sum;
            red_max[threadIdx.x >> 6] = top;
        }
        __syncthreads();
        sum = 0.0;
        top = 0.0f;
#pragma unroll
        for (int w = 0; w < NT / 64; ++w) {
            sum += red_sum[w];
            top = max_abs(top, red_max[w]);
        }
    }
}

// rows of NT < 256 threads share workgroups of 256
template <int NT>
__device__ __forceinline__ int row_of_thread() {
    return NT < 256 ? (int)(blockIdx.x * (256 / NT) + threadIdx.x / NT) : (int)blockIdx.x;
}

// ---------------------------------------------------------------------------
// rms_norm: NT threads per row, CPT 16-byte chunks per thread in registers.
// x, residual and h may be the same memory: a thread reads its elements before
// it writes them, and no other thread touches them.
// ---------------------------------------------------------------------------
struct NormArgs {
    const u32x4* x;
    const u32x4* r;          // residual or null
    const u32x4* w;
    u32x4* h;                // or null
    u32x4* y;                // or null with codes
    uint2* q;
    float* s;
    double inv_K;
    float eps;
    int M, K;
};

// The squares are summed in fp64: rows near either end of bf16's range (1e30,
// 1e-30) neither overflow nor vanish, and the result does not depend on how a
// row is split over threads.  It costs nothing visible beside the row's bytes.
//
// The scale needs max |h rstd w|.  max |h w| is known before rstd, so both
// reductions share one barrier, and the maximum is that times rstd; a row whose
// |h w| leaves the middle of fp32's range, or holds a NaN, reduces once more.
template <class Fmt, int NT, int CPT>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void rms_norm_kernel(NormArgs p) {
    constexpr int NW = NT < 256 ? 4 : NT / 64;
    __shared__ double red_sum[NW];
    __shared__ float red_max[2][NW];
    const int tid = threadIdx.x % NT;
    const int m = row_of_thread<NT>();
    if (m >= p.M) return;                                    // all threads of a row together
    const int chunks = p.K >> 3;
    const size_t row = (size_t)m * chunks;
    u32x4 xv[CPT], rv[CPT], wv[CPT];
    // with a residual this is the last use of x and of the old stream, and the new
    // one is read only after two products: all pass the caches by, at every size
    // (to bf16 / e4m3 without and with: 8191 x 8192 92.6 / 81.8 and 90.3 / 79.0 us, 1024 x
    // 8192 15.3 / 14.6 and 13.6 / 12.7, 512 x 8192 8.3 / 8.5 and 8.3 / 8.2, 256 x 4096 4.1 /
    // 4.3 and 3.9 / 4.0; 128 x 8192 4.2 / 4.6 and 4.5 / 4.4, below no difference)
    if (p.r) {
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int c = tid + i * NT;
            xv[i] = c < chunks ? load_row<true>(p.x + row + c) : u32x4{0u, 0u, 0u, 0u};
            rv[i] = c < chunks ? load_row<true>(p.r + row + c) : u32x4{0u, 0u, 0u, 0u};
        }
    } else {
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int c = tid + i * NT;
            xv[i] = c < chunks ? p.x[row + c] : u32x4{0u, 0u, 0u, 0u};
        }
    }
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        const int c = tid + i * NT;
        wv[i] = c < chunks ? p.w[c] : u32x4{0u, 0u, 0u, 0u};
    }
    float v[CPT][8];
    double sum = 0.0;
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        unpack8(xv[i], v[i]);
        if (p.r) {
            float f[8];
            unpack8(rv[i], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i][j] += f[j];
        }
        const int c = tid + i * NT;
        if (p.h && c < chunks) store_row<true>(p.h + row + c, pack8(v[i]));
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fma((double)v[i][j], (double)v[i][j], sum);
        if constexpr (kCodes<Fmt>) {
            float f[8];
            unpack8(wv[i], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) top = max_abs(top, v[i][j] * f[j]);
        }
    }
    if constexpr (kCodes<Fmt>) row_sum_max<NT>(sum, top, red_sum, red_max[0]);
    else sum = row_sum<NT>(sum, red_sum);
    const float rstd = rstd_of(sum, p.inv_K, p.eps);
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        const int c = tid + i * NT;
        float f[8];
        unpack8(wv[i], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * rstd * f[j];
        if (p.y && c < chunks) p.y[row + c] = pack8(v[i]);
    }
    if constexpr (kCodes<Fmt>) {
        if (top >= 0x1p-100f && top < __builtin_inff()) {    // uniform in the row
            top *= rstd;
        } else {
            top = 0.0f;
#pragma unroll
            for (int i = 0; i < CPT; ++i)
#pragma unroll
                for (int j = 0; j < 8; ++j) top = max_abs(top, v[i][j]);
            top = row_max<NT>(top, red_max[1]);
        }
        const RowScale sc = RowScale::of<Fmt>(top);
        if (tid == 0) p.s[m] = sc.s;
#pragma unroll
        for (int i = 0; i < CPT; ++i) {
            const int c = tid + i * NT;
            if (c < chunks) p.q[row + c] = sc.codes<Fmt>(v[i]);
        }
    }
}

// Rows too long for registers: the row is read again for every step (h last, so
// that it may overwrite x or the residual).
template <class Fmt>
__global__ __launch_bounds__(1024) void rms_norm_long_kernel(NormArgs p) {
    constexpr int NT = 1024;
    __shared__ double red_sum[NT / 64];
    __shared__ float red_max[NT / 64];
    const int tid = threadIdx.x;
    const int m = blockIdx.x;
    const int chunks = p.K >> 3;
    const size_t row = (size_t)m * chunks;
    auto load = [&](int c, float* v) {
        unpack8(p.x[row + c], v);
        if (p.r) {
            float f[8];
            unpack8(p.r[row + c], f);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] += f[j];
        }
    };
    double sum = 0.0;
    for (int c = tid; c < chunks; c += NT) {
        float v[8];
        load(c, v);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum = fma((double)v[j], (double)v[j], sum);
    }
    const float rstd = rstd_of(row_sum<NT>(sum, red_sum), p.inv_K, p.eps);
    auto norm = [&](int c, float* v) {
        float f[8];
        unpack8(p.w[c], f);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = v[j] * rstd * f[j];
    };
    RowScale sc{};
    if constexpr (kCodes<Fmt>) {
        float amax = 0.0f;
        for (int c = tid; c < chunks; c += NT) {
            float v[8];
            load(c, v);
            norm(c, v);
#pragma unroll
            for (int j = 0; j < 8; ++j) amax = max_abs(amax, v[j]);
        }
        sc = RowScale::of<Fmt>(row_max<NT>(amax, red_max));
        if (tid == 0) p.s[m] = sc.s;
    }
    for (int c = tid; c < chunks; c += NT) {
        float v[8];
        load(c, v);
        if (p.h) p.h[row + c] = pack8(v);
        norm(c, v);
        if (p.y) p.y[row + c] = pack8(v);
        if constexpr (kCodes<Fmt>) p.q[row + c] = sc.codes<Fmt>(v);
    }
}

// Threads per row and chunks per thread of a row of `chunks` pieces: part of a
// wave up to 32 pieces (norm to e4m3 at 16384 x 128 6.0 us, with a whole wave a
// row 11.7), one wave up to 128, else one workgroup with two to four chunks a
// thread (measured against one chunk and 1024 threads, and against eight: norm to
// e4m3 at 8191 x 8192 79 us, 91 and 80, at 1024 x 8192 12.7, 15.0 and 14.2; swiglu to
// e4m3 at 8192 x 4096 28 us with 256 threads, 37 with 512).  `many` (coded rows, four
// a CU or more): one wave up to 256 pieces, which saves the barriers (swiglu at
// 16384 x 2048 29 us against 34; with few rows a CU holds too few waves; the bf16
// norm, with one barrier, gains nothing).
template <class Go>
static bool with_row_shape(int chunks, bool many, Go&& go) {
    if (chunks <= 8) go(ic<8>{}, ic<1>{});
    else if (chunks <= 16) go(ic<16>{}, ic<1>{});
    else if (chunks <= 32) go(ic<32>{}, ic<1>{});
    else if (chunks <= 64) go(ic<64>{}, ic<1>{});
    else if (chunks <= 128) go(ic<64>{}, ic<2>{});
    else if (chunks <= 192 && many) go(ic<64>{}, ic<3>{});
    else if (chunks <= 256 && many) go(ic<64>{}, ic<4>{});
    else if (chunks <= 256) go(ic<256>{}, ic<1>{});
    else if (chunks <= 512) go(ic<256>{}, ic<2>{});
    else if (chunks <= 1024) go(ic<512>{}, ic<2>{});
    else if (chunks <= 2048) go(ic<512>{}, ic<4>{});
    else if (chunks <= 4096) go(ic<1024>{}, ic<4>{});
    else return false;
    return true;
}
static bool many_rows(int M) { return M >= 4 * device_cu_count(); }
// workgroups and threads of M rows at NT threads a row
template <int NT>
static dim3 row_grid(int M) { return dim3(NT < 256 ? (M + 256 / NT - 1) / (256 / NT) : M); }
template <int NT>
static dim3 row_block() { return dim3(NT < 256 ? 256 : NT); }

template <class Fmt>
static void launch_norm(const NormArgs& p, hipStream_t st) {
    const bool done = with_row_shape(p.K / 8, kCodes<Fmt> && many_rows(p.M), [&](auto nt, auto cpt) {
        constexpr int NT = decltype(nt)::value, CPT = decltype(cpt)::value;
        hipLaunchKernelGGL((rms_norm_kernel<Fmt, NT, CPT>), row_grid<NT>(p.M), row_block<NT>(), 0, st, p);
    });
    if (!done) hipLaunchKernelGGL(rms_norm_long_kernel<Fmt>, dim3(p.M), dim3(1024), 0, st, p);
}

void launch_rms_norm(const uint16_t* x, const uint16_t* r, const uint16_t* w, float eps, int M, int K, uint16_t* h,
                     uint16_t* y, void* q, float* s, ActFormat fmt, hipStream_t st) {
    const NormArgs p{reinterpret_cast<const u32x4*>(x), reinterpret_cast<const u32x4*>(r),
                     reinterpret_cast<const u32x4*>(w), reinterpret_cast<u32x4*>(h), reinterpret_cast<u32x4*>(y),
                     static_cast<uint2*>(q), s, 1.0 / K, eps, M, K};
    if (fmt == ActFormat::bf16) launch_norm<FmtNone>(p, st);
    else if (fmt == ActFormat::e4m3) launch_norm<FmtE4M3>(p, st);
    else launch_norm<FmtI8>(p, st);
}

// ---------------------------------------------------------------------------
// swiglu on the fused gate_up output [M, 2I]: gate in the first I columns.
// ---------------------------------------------------------------------------
struct SwigluArgs {
    const u32x4* gu;
    u32x4* y;                // bf16 output
    uint2* q;
    float* s;
    int M, I;
};

// silu(g) u = g u / (1 + 2^(-g log2 e)) on the hardware's 2^t and reciprocal (one
// unit in the last place each); the rounding of t adds |g| 2^-24 to the relative
// error where the exponential dominates (g < 0).  A gate below -87 makes the
// denominator infinite or its reciprocal vanish: the product is then -0, off by
// less than 2^-126 |g u|.
__device__ __forceinline__ void swiglu8(u32x4 gate, u32x4 up, float* y) {
    float g[8], u[8];
    unpack8(gate, g);
    unpack8(up, u);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        y[j] = g[j] * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-1.44269504f * g[j])) * u[j];
}

// STREAM: the gate_up output, dead after this, passes the caches by (8192 x 14336
// to bf16 / e4m3 121 / 109 us without, 116 / 103 with, 16384 x 2048 36 / 33 and 34 / 29;
// 256 x 14336, which the L2s hold, 5.2 / 6.1 without, 5.5 / 6.3 with).
static bool stream_gate_up(const SwigluArgs& p) { return (size_t)p.M * p.I * 4 > kStreamBytes; }

// no row reduction: the grid covers the chunks of all rows
template <bool STREAM>
__global__ __launch_bounds__(256) void swiglu_kernel(SwigluArgs p) {
    const int chunks = p.I >> 3;
    const uint32_t i = blockIdx.x * 256u + threadIdx.x;      // a dispatch holds fewer than 2^32 threads
    const uint32_t m = i / (uint32_t)chunks;
    if (m >= (uint32_t)p.M) return;
    const u32x4* gate = p.gu + i + (size_t)m * chunks;
    float y[8];
    swiglu8(load_row<STREAM>(gate), load_row<STREAM>(gate + chunks), y);
    p.y[i] = pack8(y);
}

template <class Fmt, int NT, int CPT, bool STREAM>
__global__ __launch_bounds__(NT < 256 ? 256 : NT) void swiglu_quant_kernel(SwigluArgs p) {
    __shared__ float red[NT < 256 ? 4 : NT / 64];
    const int tid = threadIdx.x % NT;
    const int m = row_of_thread<NT>();
    if (m >= p.M) return;
    const int chunks = p.I >> 3;
    const u32x4* gate = p.gu + (size_t)m * 2 * chunks;
    u32x4 g[CPT], u[CPT];
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        const int c = tid + i * NT;
        g[i] = u[i] = u32x4{0u, 0u, 0u, 0u};
        if (c < chunks) {
            g[i] = load_row<STREAM>(gate + c);
            u[i] = load_row<STREAM>(gate + chunks + c);
        }
    }
    float y[CPT][8];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        swiglu8(g[i], u[i], y[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = max_abs(amax, y[i][j]);
    }
    const RowScale sc = RowScale::of<Fmt>(row_max<NT>(amax, red));
    if (tid == 0) p.s[m] = sc.s;
#pragma unroll
    for (int i = 0; i < CPT; ++i) {
        const int c = tid + i * NT;
        if (c < chunks) p.q[(size_t)m * chunks + c] = sc.codes<Fmt>(y[i]);
    }
}

template <class Fmt>
__global__ __launch_bounds__(1024) void swiglu_quant_long_kernel(SwigluArgs p) {
    constexpr int NT = 1024;
    __shared__ float red[NT / 64];
    const int m = blockIdx.x;
    const int chunks = p.I >> 3;
    const u32x4* gate = p.gu + (size_t)m * 2 * chunks;
    float amax = 0.0f;
    for (int c = threadIdx.x; c < chunks; c += NT) {
        float y[8];
        swiglu8(gate[c], gate[chunks + c], y);
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = max_abs(amax, y[j]);
    }
    const RowScale sc = RowScale::of<Fmt>(row_max<NT>(amax, red));
    if (threadIdx.x == 0) p.s[m] = sc.s;
    for (int c = threadIdx.x; c < chunks; c += NT) {
        float y[8];
        swiglu8(gate[c], gate[chunks + c], y);
        p.q[(size_t)m * chunks + c] = sc.codes<Fmt>(y);
    }
}

template <class Fmt>
static void launch_swiglu_quant(const SwigluArgs& p, hipStream_t st) {
    const bool done = with_row_shape(p.I / 8, many_rows(p.M), [&](auto nt, auto cpt) {
        constexpr int NT = decltype(nt)::value, CPT = decltype(cpt)::value;
        if (stream_gate_up(p))
            hipLaunchKernelGGL((swiglu_quant_kernel<Fmt, NT, CPT, true>), row_grid<NT>(p.M), row_block<NT>(), 0, st, p);
        else
            hipLaunchKernelGGL((swiglu_quant_kernel<Fmt, NT, CPT, false>), row_grid<NT>(p.M), row_block<NT>(), 0, st, p);
    });
    if (!done) hipLaunchKernelGGL(swiglu_quant_long_kernel<Fmt>, dim3(p.M), dim3(1024), 0, st, p);
}

void launch_swiglu(const uint16_t* gu, int M, int I, uint16_t* y, void* q, float* s, ActFormat fmt, hipStream_t st) {
    const SwigluArgs p{reinterpret_cast<const u32x4*>(gu), reinterpret_cast<u32x4*>(y), static_cast<uint2*>(q), s, M, I};
    if (fmt == ActFormat::e4m3) {
        launch_swiglu_quant<FmtE4M3>(p, st);
    } else if (fmt == ActFormat::int8) {
        launch_swiglu_quant<FmtI8>(p, st);
    } else {
        const size_t total = (size_t)M * (I / 8);
        const dim3 grid((unsigned)((total + 255) / 256));
        if (stream_gate_up(p)) hipLaunchKernelGGL(swiglu_kernel<true>, grid, dim3(256), 0, st, p);
        else hipLaunchKernelGGL(swiglu_kernel<false>, grid, dim3(256), 0, st, p);
    }
}

}  // namespace qg
