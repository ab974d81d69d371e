// Between the qkv product and attention: the RMS norm of every query and key head, the
// rotation by position, and the keys' and values' way into a paged cache, in one pass
// over the product's output.
//
//   y = (x * rsqrt(mean(x^2) + eps)) * weight              per head, or y = x
//   (y_a, y_b) <- (y_a cos - y_b sin, y_b cos + y_a sin)    angle = position * inv_freq[i]
//       half-split pairs (i, i + R / 2) or neighbours (2 i, 2 i + 1), i < R / 2
//
// fp32 from the bf16 inputs to the one rounding of each output; squares whose fp32 sum
// leaves [2^-80, 2^100] are summed in fp64 (rows near 1e+-30 stay finite).  Angles are
// fp64 turns: position * inv_freq / (2 pi), less its nearest whole number, is exact to
// 2^-22 turns at any 32-bit position and feeds the hardware's sine and cosine of turns
// (1.3e-7 absolute over a whole turn).
// No table of angles: positions have no limit, and a token's 64 angles cost less than
// reading them.
//
// A lane holds eight neighbouring elements of a head (16 bytes), D / 8 lanes a head.  A token's
// heads are taken by one wave, or dealt to several while those are few (`launch`): in each, a lane
// computes one pair's angle and the heads' lanes read theirs from LDS (every lane its own eight
// took 4 KB of frequencies a wave, 78 us instead of 65 at 8191 tokens).  A pair's other half is
// read again from the L1 rather than moved between lanes.
// Bound by memory: 8191 tokens of 64 + 8 heads, normed, 65 us (4.7 TB/s; a copy 5.2); a
// head at a time and 8 waves a SIMD beat two or four heads at a time and fewer (71 / 81 us).

#include <algorithm>

#include "codes.h"
#include "device_common.h"
#include "launch.h"
#include "rows.h"
#include "sequences.h"

namespace qg {

namespace {

enum class To { dense, cache_bf16, cache_e4m3 };
enum class Kind { query, key, value };

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

// Multiplies a head's x and its pairs' halves y by the norm's factor 1 / sqrt(mean(x^2) + eps):
// before the weight, with which either may leave fp32's range though their quotient's product
// does not.  Squares and sum are fp32 where that neither overflows nor loses the small ones (all
// rows but extreme ones), else fp64.
template <int L>
__device__ __forceinline__ void norm_head(float* x, float* y, double inv_D, float eps) {
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < 8; ++j) sum = fmaf(x[j], x[j], sum);
    sum = head_sum<L>(sum);
    float r;
    if (sum >= 0x1p-80f && sum <= 0x1p100f) {
        const float v = fmaf(sum, (float)inv_D, eps);
        r = __builtin_amdgcn_rsqf(v);
        r = fmaf(r * 0.5f, fmaf(-v * r, r, 1.0f), r);
    } else {
        double wide = 0.0;
#pragma unroll
        for (int j = 0; j < 8; ++j) wide = fma((double)x[j], (double)x[j], wide);
        r = rstd_of(head_sum<L>(wide), inv_D, eps);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        x[j] *= r;
        y[j] *= r;
    }
}

// Where a token's key and value go: a row of the cache, or nowhere (-1).
__device__ __forceinline__ int64_t cache_row(const RopeArgs& p, int b, int pos) {
    if (b < 0 || pos < 0 || (pos >> p.page_shift) >= p.max_pages) return -1;
    const int page = p.table[(int64_t)b * p.max_pages + (pos >> p.page_shift)];
    if (page < 0 || page >= p.pages) return -1;
    return (((int64_t)page * p.Hkv) << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
}

// NEXT: pairs of neighbours, else (i, i + rot / 2)
template <int D, To TO, bool NEXT>
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
    const int half = p.rot >> 1, d0 = piece * 8;
    const bool turns = d0 < p.rot, upper = !NEXT && d0 >= half;
    const int other = !turns || NEXT ? piece : upper ? piece - half / 8 : piece + half / 8;
    // an angle a lane (at most 64 pairs), handed to the lanes of every head through LDS
    __shared__ __attribute__((aligned(16))) float table[4][2][64];
    float (*angles)[64] = table[threadIdx.x >> 6];
    if (lane < half) {
        double turn = (double)pos * p.inv_freq[lane] * 0.15915494309189533577;    // 1 / (2 pi)
        turn -= rint(turn);
        angles[0][lane] = __builtin_amdgcn_cosf((float)turn);
        angles[1][lane] = __builtin_amdgcn_sinf((float)turn);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    // this lane's factors of x and of `other` (its sign in the second)
    auto factors = [&](float* c, float* s) {
#pragma unroll
        for (int j = 0; j < 8; ++j) c[j] = 1.0f, s[j] = 0.0f;
        if (!turns) return;
        const int at = NEXT ? d0 / 2 : upper ? d0 - half : d0;
        float cos[8], sin[8];
#pragma unroll
        for (int i = 0; i < (NEXT ? 4 : 8); i += 4) {
            *reinterpret_cast<f32x4*>(cos + i) = *reinterpret_cast<const f32x4*>(angles[0] + at + i);
            *reinterpret_cast<f32x4*>(sin + i) = *reinterpret_cast<const f32x4*>(angles[1] + at + i);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            c[j] = cos[NEXT ? j / 2 : j];
            s[j] = (NEXT ? j & 1 : upper) ? sin[NEXT ? j / 2 : j] : -sin[NEXT ? j / 2 : j];
        }
    };

    const u32x4* in = reinterpret_cast<const u32x4*>(p.qkv) + (int64_t)t * (p.Hq + 2 * p.Hkv) * L;
    // The query, key and value heads in turn, HS at a time, dealt to the token's waves.
    int dealt = 0;
    auto heads = [&](auto kind, int h0, int H, const uint16_t* weight) {
        constexpr Kind KIND = decltype(kind)::value;
        const int units = (H + HS - 1) / HS, parts = 1 << p.parts_shift;
        const int first = (part - dealt) & (parts - 1);
        dealt += units;
        if (first >= units) return;
        const bool moves = KIND != Kind::value && turns;
        // the norm's weight goes into the pair's factors (a factor of each half)
        float cg[8], sg[8];
        const bool norm = KIND != Kind::value && weight;
        if (KIND != Kind::value) factors(cg, sg);
        if (norm) {
            float g[8], g2[8];
            unpack8(reinterpret_cast<const u32x4*>(weight)[piece], g);
            unpack8(reinterpret_cast<const u32x4*>(weight)[other], g2);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                cg[j] *= g[j];
                sg[j] *= NEXT ? g[j ^ 1] : g2[j];
            }
        }
        for (int u = first; u < units; u += parts) {
            const int h = u * HS + lane / L;
            if (h >= H) continue;
            u32x4 packed = in[(h0 + h) * L + piece];
            float x[8];
            unpack8(packed, x);
            if (KIND != Kind::value && (moves || norm)) {
                float y[8];
                unpack8(NEXT ? packed : in[(h0 + h) * L + other], y);
                if (norm) norm_head<L>(x, y, 1.0 / D, p.eps);
                if (moves) {
                    if constexpr (NEXT) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) y[j] = x[j ^ 1];
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] = fmaf(y[j], sg[j], x[j] * cg[j]);
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) x[j] *= cg[j];
                }
                packed = pack8(x);
            }
            if constexpr (KIND == Kind::query) {
                reinterpret_cast<u32x4*>(p.q)[((int64_t)t * p.Hq + h) * L + piece] = packed;
            } else if constexpr (TO == To::dense) {
                reinterpret_cast<u32x4*>(p.k_dense)[((int64_t)t * p.Hkv + h) * L + piece] = packed;
            } else {
                if (row < 0) continue;
                const int64_t at = row + ((int64_t)h << p.page_shift);
                if constexpr (TO == To::cache_bf16) {
                    static_cast<u32x4*>(KIND == Kind::key ? p.k : p.v)[at * L + piece] = packed;
                } else {
                    float top = 0.0f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) top = max_abs(top, x[j]);
                    const RowScale scale = RowScale::of<FmtE4M3>(head_max<L>(top));
                    static_cast<uint2*>(KIND == Kind::key ? p.k : p.v)[at * L + piece] = scale.codes<FmtE4M3, true>(x);
                    if (piece == 0) (KIND == Kind::key ? p.k_scale : p.v_scale)[at] = scale.s;
                }
            }
        }
    };
    heads(std::integral_constant<Kind, Kind::query>{}, 0, p.Hq, p.wq);
    heads(std::integral_constant<Kind, Kind::key>{}, p.Hq, p.Hkv, p.wk);
    if constexpr (TO != To::dense) heads(std::integral_constant<Kind, Kind::value>{}, p.Hq + p.Hkv, p.Hkv, nullptr);
}

template <int D>
void launch(RopeArgs p, To to, hipStream_t st) {
    constexpr int HS = 512 / D;
    const int units = (p.Hq + HS - 1) / HS + (p.Hkv + HS - 1) / HS * (to == To::dense ? 1 : 2);
    // Waves a token: up to 8192 of them (8 a SIMD) while its heads keep them busy, and two up to 16384
    // tokens.  1000 tokens of 72 heads: 8 waves each 8.5 us, 16 10.9; 8191: one 69.6, two 64.9, four 77.
    p.parts_shift = 0;
    while ((1 << p.parts_shift) < units && (int64_t(p.T) << (p.parts_shift + 1)) <= 8192) ++p.parts_shift;
    if (p.parts_shift == 0 && units > 1 && p.T < 16384) p.parts_shift = 1;
    const dim3 grid((unsigned)(((int64_t(p.T) << p.parts_shift) + 3) / 4));
    auto run = [&](auto next) {
        constexpr bool NEXT = decltype(next)::value;
        if (to == To::dense) rope_kernel<D, To::dense, NEXT><<<grid, 256, 0, st>>>(p);
        else if (to == To::cache_bf16) rope_kernel<D, To::cache_bf16, NEXT><<<grid, 256, 0, st>>>(p);
        else rope_kernel<D, To::cache_e4m3, NEXT><<<grid, 256, 0, st>>>(p);
    };
    if (p.interleaved) run(std::true_type{});
    else run(std::false_type{});
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
