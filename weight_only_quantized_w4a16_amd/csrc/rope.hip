// Between the qkv product and attention: the RMS norm of every query and key head, the
// rotation by position, and the keys' and values' way into a paged cache, in one pass
// over the product's output.
//
//   y = (x * rsqrt(mean(x^2) + eps)) * weight              per head, or y = x
//   (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin)    angle = position * inv_freq[i]
//       half-split pairs (i, i + R / 2) or neighbours (2 i, 2 i + 1), i < R / 2
//
// fp32 from the bf16 inputs to the one rounding of each output, the squares summed in
// fp64 (rows near 1e+-30 stay finite).  Angles are fp64 turns: position * inv_freq /
// (2 pi), less its nearest whole number, is exact to 2^-22 turns at any 32-bit position
// and feeds the hardware's sine and cosine of turns (1.3e-7 absolute over a whole turn).
// No table of angles: positions have no limit, and a token's 64 angles cost less than
// reading them.
//
// A lane holds eight neighbouring elements of a head (16 bytes), D / 8 lanes a head; its
// angles stay in registers while its wave goes over the heads of its token.  A pair's
// other half is read again from the caches rather than moved between lanes.

#include <algorithm>

#include "codes.h"
#include "device_common.h"
#include "launch.h"
#include "rows.h"
#include "sequences.h"

namespace qg {

namespace {

enum class To { dense, cache_bf16, cache_e4m3 };

// Sum and largest magnitude over the L = 8 or 16 lanes of a head, in every lane.
template <int L, class T>
__device__ __forceinline__ T head_sum(T v) {
    v += dpp<0xb1>(v);                               // lane ^ 1
    v += dpp<0x4e>(v);                               // lane ^ 2
    v += dpp<0x141>(v);                              // the other four of eight
    if constexpr (L == 16) v += dpp<0x140>(v);       // the other eight of sixteen
    return v;
}
// for a >= 0 or NaN: their bits order as the values do
template <int L>
__device__ __forceinline__ float head_max(float a) {
    uint32_t u = __float_as_uint(a) & 0x7fffffffu;
    u = max(u, dpp_u32<0xb1>(0u, u));
    u = max(u, dpp_u32<0x4e>(0u, u));
    u = max(u, dpp_u32<0x141>(0u, u));
    if constexpr (L == 16) u = max(u, dpp_u32<0x140>(0u, u));
    return __uint_as_float(u);
}

// Where a token's key and value go: a row of the cache, or nowhere (-1).
__device__ __forceinline__ int64_t cache_row(const RopeArgs& p, int b, int pos) {
    if (b < 0 || pos < 0 || (pos >> p.page_shift) >= p.max_pages) return -1;
    const int page = p.table[(int64_t)b * p.max_pages + (pos >> p.page_shift)];
    if (page < 0 || page >= p.pages) return -1;
    return (((int64_t)page * p.Hkv) << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
}

template <int D, To TO>
__global__ __launch_bounds__(256) void rope_kernel(RopeArgs p) {
    constexpr int L = D / 8;                         // lanes of a head
    constexpr int HS = 64 / L;                       // heads of a wave at a time
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane((int)(blockIdx.x * 4 + (threadIdx.x >> 6)));
    const int t = wave >> p.parts_shift;             // 2^parts_shift waves a token
    if (t >= p.T) return;
    const int part = wave & ((1 << p.parts_shift) - 1);
    const int piece = lane & (L - 1);
    int pos;
    int64_t row = -1;
    if constexpr (TO == To::dense) {
        pos = p.positions[t];
    } else {
        const int b = sequence_of_token(p.q_offsets, p.B, t);
        if (b < 0) return;                           // behind the last sequence: left as it is
        const Sequence s = sequence_of(p.q_offsets[b], p.q_offsets[b + 1], p.kv_len[b], p.T);
        pos = s.len - s.tokens + (t - s.first_token);
        row = cache_row(p, b, pos);
    }

    // out = x * c + other * s, `other` being the pair's other half with its sign in s
    const int half = p.rot >> 1;
    const bool turns = piece * 8 < p.rot;
    float c[8], s[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) c[j] = 1.0f, s[j] = 0.0f;
    int other = piece;
    if (turns) {
        const int d0 = piece * 8;
        const bool upper = !p.interleaved && d0 >= half;
        if (!p.interleaved) other = upper ? piece - half / 8 : piece + half / 8;
        const double* f = p.inv_freq + (p.interleaved ? d0 / 2 : upper ? d0 - half : d0);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (p.interleaved && (j & 1)) {
                c[j] = c[j - 1];
                s[j] = -s[j - 1];
                continue;
            }
            double turn = (double)pos * f[p.interleaved ? j / 2 : j] * 0.15915494309189533577;    // 1 / (2 pi)
            turn -= rint(turn);
            const float x = (float)turn;
            c[j] = __builtin_amdgcn_cosf(x);
            s[j] = __builtin_amdgcn_sinf(x);
            if (!upper) s[j] = -s[j];
        }
    }

    const int rotated = p.Hq + p.Hkv;
    const int heads = TO == To::dense ? rotated : rotated + p.Hkv;
    const u32x4* in = reinterpret_cast<const u32x4*>(p.qkv) + (int64_t)t * (p.Hq + 2 * p.Hkv) * L;
    for (int h = part * HS + lane / L; h < heads; h += HS << p.parts_shift) {
        const u32x4 raw = in[h * L + piece];
        const bool moves = turns && h < rotated;
        u32x4 raw2 = raw;
        if (moves && !p.interleaved) raw2 = in[h * L + other];
        float x[8];
        unpack8(raw, x);
        u32x4 packed = raw;
        const u32x4* w = reinterpret_cast<const u32x4*>(h < p.Hq ? p.wq : h < rotated ? p.wk : nullptr);
        if (moves || w) {
            float y[8];
            unpack8(raw2, y);
            if (w) {
                double sum = 0.0;
#pragma unroll
                for (int j = 0; j < 8; ++j) sum = fma((double)x[j], (double)x[j], sum);
                const float r = rstd_of(head_sum<L>(sum), 1.0 / D, p.eps);
                float g[8];
                unpack8(w[piece], g);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = x[j] * r * g[j];
                if (moves && !p.interleaved) {
                    unpack8(w[other], g);
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] = y[j] * r * g[j];
                }
            }
            if (moves) {
                if (p.interleaved) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) y[j] = x[j ^ 1];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] = fmaf(y[j], s[j], x[j] * c[j]);
            }
            packed = pack8(x);
        }
        if (h < p.Hq) {
            reinterpret_cast<u32x4*>(p.q)[((int64_t)t * p.Hq + h) * L + piece] = packed;
            continue;
        }
        const int hk = h < rotated ? h - p.Hq : h - rotated;
        if constexpr (TO == To::dense) {
            reinterpret_cast<u32x4*>(p.k_dense)[((int64_t)t * p.Hkv + hk) * L + piece] = packed;
        } else {
            if (row < 0) continue;
            const int64_t at = row + ((int64_t)hk << p.page_shift);
            if constexpr (TO == To::cache_bf16) {
                static_cast<u32x4*>(h < rotated ? p.k : p.v)[at * L + piece] = packed;
            } else {
                float top = 0.0f;
#pragma unroll
                for (int j = 0; j < 8; ++j) top = max_abs(top, x[j]);
                const RowScale scale = RowScale::of<FmtE4M3>(head_max<L>(top));
                static_cast<uint2*>(h < rotated ? p.k : p.v)[at * L + piece] = scale.codes<FmtE4M3>(x);
                if (piece == 0) (h < rotated ? p.k_scale : p.v_scale)[at] = scale.s;
            }
        }
    }
}

template <int D>
void launch(RopeArgs p, To to, hipStream_t st) {
    constexpr int HS = 512 / D;
    const int heads = p.Hq + p.Hkv + (to == To::dense ? 0 : p.Hkv);
    const int units = (heads + HS - 1) / HS;
    // waves a token: as many as its heads keep busy while the tokens alone do not fill the GPU
    p.parts_shift = 0;
    while ((1 << p.parts_shift) < units && (int64_t(p.T) << p.parts_shift) < 8192) ++p.parts_shift;
    const dim3 grid((unsigned)(((int64_t(p.T) << p.parts_shift) + 3) / 4));
    if (to == To::dense) rope_kernel<D, To::dense><<<grid, 256, 0, st>>>(p);
    else if (to == To::cache_bf16) rope_kernel<D, To::cache_bf16><<<grid, 256, 0, st>>>(p);
    else rope_kernel<D, To::cache_e4m3><<<grid, 256, 0, st>>>(p);
}

void launch(const RopeArgs& p, int D, To to, hipStream_t st) {
    if (D == 64) launch<64>(p, to, st);
    else launch<128>(p, to, st);
}

}  // namespace

void launch_qk_norm_rope(const RopeArgs& p, int D, hipStream_t st) { launch(p, D, To::dense, st); }
void launch_kv_append(const RopeArgs& p, int D, hipStream_t st) {
    launch(p, D, p.k_scale ? To::cache_e4m3 : To::cache_bf16, st);
}

}  // namespace qg
