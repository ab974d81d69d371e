// The way into and out of the expert-grouped products: B tokens with k chosen
// experts each make T = B k slots; the slots, sorted by expert (stable: slot
// order inside an expert), are the routed rows.
//
//   dispatch  offsets[e] = first row of expert e, row_of_slot[b, j] = the row of
//             slot (b, j), out[row_of_slot[b, j]] = rows[b]
//   combine   y[b] = sum_j w[b, j] rows[row_of_slot[b, j]] + residual[b], fp32
//   gradient  drows[row_of_slot[b, j]] = w[b, j] dy[b],
//             dw[b, j] = <dy[b], rows[row_of_slot[b, j]]>
//
// A slot whose expert id lies outside [0, E) has no row (row_of_slot = -1) and
// takes part in nothing.  Every kernel works by token: a token's row is read
// once however many experts chose it, and its k routed rows meet in registers
// in slot order, so no atomics and no second order of summation exist.  All of
// them are bound by memory from about a thousand tokens on, by the launch below.
// Graph-timed, on buffers in turn that no cache holds (top-8 of 128, rows of 2048,
// 8192 / 64 / 1 tokens, us): dispatch of e4m3 rows 38 / 4.5 / 3.8 (4.0 TB/s at 8192),
// combine of bf16 rows 60 / 3.3 / 2.7 (5.6 TB/s), its gradient 108 / 4.4 / 3.8 (5.3 TB/s).
#include <algorithm>
#include <atomic>

#include "device_common.h"
#include "launch.h"
#include "rows.h"

namespace qg {

// ---------------------------------------------------------------------------
// The sort of many slots: a counting sort in two launches.  Segment i of the
// slots (one workgroup, `seg` slots) counts its experts into hist[i][e]; then
// every segment derives the first row of each expert (totals over all segments)
// and of its own share (totals over the segments before it), and numbers its
// slots in order.  The work is latency, not bandwidth: up to SORT_MAX_SEGS segments
// hold one slot per thread (REG), beyond that they grow and are read twice
// (measured, one / two / four slots per thread, 128 experts, us: 8192 slots 6.3 /
// 7.1 / 8.2, 65536 6.9 / 8.2 / 9.1, 262144 9.3 / 8.6 / 9.3).
// ---------------------------------------------------------------------------
constexpr int SORT_WAVES = 16;
constexpr int SORT_NT = SORT_WAVES * 64;
constexpr int SORT_MAX_SEGS = 256;

// slots per segment, a multiple of SORT_NT
static int sort_seg(int T) {
    const int seg = (T + SORT_MAX_SEGS - 1) / SORT_MAX_SEGS;
    return (seg + SORT_NT - 1) / SORT_NT * SORT_NT;
}

__global__ __launch_bounds__(SORT_NT) void moe_count_kernel(const int* __restrict__ ids, int T, int E, int seg,
                                                            int* __restrict__ hist) {
    extern __shared__ int count[];               // [E]
    for (int e = threadIdx.x; e < E; e += SORT_NT) count[e] = 0;
    __syncthreads();
    const int s0 = blockIdx.x * seg;
    const int s1 = min(s0 + seg, T);
    for (int s = s0 + (int)threadIdx.x; s < s1; s += SORT_NT) {
        const int e = ids[s];
        if (e >= 0 && e < E) atomicAdd(&count[e], 1);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += SORT_NT) hist[(size_t)blockIdx.x * E + e] = count[e];
}

// lanes of the wave whose `key` (below 2^bits) equals this lane's, among `live`
__device__ __forceinline__ uint64_t same_key(int key, int bits, uint64_t live) {
    uint64_t m = live;
    for (int b = 0; b < bits; ++b) {
        const uint64_t one = __ballot((key >> b) & 1);
        m &= ((key >> b) & 1) ? one : ~one;
    }
    return m;
}

// Exclusive scan over the experts of the totals all[e] in LDS by a workgroup of
// NW waves (E <= 1024): first[e] = sum of all[0 .. e-1]; offsets, if given, too.
template <int NW>
__device__ __forceinline__ void scan_experts(const int* all, int E, int* first, int* offsets, int* wave_total) {
    const int lane = threadIdx.x & 63;
    const int wave = threadIdx.x >> 6;
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += NW * 64) {
        const int e = e0 + (int)threadIdx.x;
        const int own = e < E ? all[e] : 0;
        int incl = own;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int v = __shfl_up(incl, d, 64);
            if (lane >= d) incl += v;
        }
        if (lane == 63) wave_total[wave] = incl;
        __syncthreads();
        int base = carry;
        for (int w = 0; w < NW; ++w) {
            base += w < wave ? wave_total[w] : 0;
            carry += wave_total[w];
        }
        if (e < E) {
            if (first) first[e] = base + incl - own;
            if (offsets) offsets[e + 1] = base + incl;
        }
        __syncthreads();                         // wave_total is written again
    }
    if (offsets && threadIdx.x == 0) offsets[0] = 0;
}

// LDS words of moe_place_kernel
static int place_words(int E) { return (2 + SORT_WAVES) * E; }

template <bool REG>
__global__ __launch_bounds__(SORT_NT) void moe_place_kernel(const int* __restrict__ ids, int T, int E, int bits, int seg,
                                                            const int* __restrict__ hist, int* __restrict__ offsets,
                                                            int* __restrict__ row_of_slot) {
    extern __shared__ int lds[];
    int* all = lds;                              // [E]: slots of the expert
    int* first = lds + E;                        // [E]: its slots in the segments before, then its first row
    int* next = lds + 2 * E;                     // [SORT_WAVES][E]: counts by wave, then the next row past `first`
    __shared__ int wave_total[SORT_WAVES];
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = tid >> 6;
    const int nseg = gridDim.x;
    const int mine = blockIdx.x;

    // each wave numbers a contiguous part of the segment, 64 slots at a time
    const int per = seg / SORT_WAVES;
    const int s0 = mine * seg + wave * per;
    const int s1 = min(s0 + per, T);
    const int held = REG && s0 + lane < s1 ? ids[s0 + lane] : -1;

    // totals over the segments: SORT_NT / 2^bits threads share an expert's column
    // (up to 2^10 experts: one thread each at least)
    for (int i = tid; i < SORT_WAVES * E; i += SORT_NT) next[i] = 0;
    for (int e = tid; e < 2 * E; e += SORT_NT) lds[e] = 0;   // all, and first as the count of the segments before
    __syncthreads();
    {
        const int e = tid & ((1 << bits) - 1);
        const int part = tid >> bits;
        const int parts = SORT_NT >> bits;
        if (e < E) {
            int total = 0, before = 0;
#pragma unroll 8
            for (int i = part; i < nseg; i += parts) {
                const int c = hist[(size_t)i * E + e];
                total += c;
                before += i < mine ? c : 0;
            }
            atomicAdd(&all[e], total);
            atomicAdd(&first[e], before);
        }
    }
    // meanwhile each wave counts its part
    int* cnt = next + wave * E;
    auto count = [&](int e) {
        if (e >= 0 && e < E) atomicAdd(&cnt[e], 1);
    };
    if constexpr (REG) {
        count(held);
    } else {
        for (int s = s0 + lane; s < s1; s += 64) count(ids[s]);
    }
    __syncthreads();
    // counts become the number of the expert's slots before each wave's
    for (int e = tid; e < E; e += SORT_NT) {
        int at = first[e];
        for (int w = 0; w < SORT_WAVES; ++w) {
            const int c = next[w * E + e];
            next[w * E + e] = at;
            at += c;
        }
    }
    __syncthreads();
    scan_experts<SORT_WAVES>(all, E, first, mine == 0 ? offsets : nullptr, wave_total);
    auto number = [&](int s, int e) {            // all lanes of the wave; s: the first lane's slot
        const bool kept = e >= 0 && e < E;
        const uint64_t live = __ballot(kept);
        const uint64_t m = same_key(kept ? e : 0, bits, live);
        int row = -1;
        int at = 0;
        if (kept) {
            at = cnt[e];
            row = first[e] + at + __popcll(m & ((1ull << lane) - 1));
        }
        __builtin_amdgcn_wave_barrier();         // every lane has read before one writes
        if (kept && (m >> lane) == 1ull) cnt[e] = at + __popcll(m);   // the last lane of each key
        __builtin_amdgcn_wave_barrier();
        if (s + lane < s1) row_of_slot[s + lane] = row;
    };
    if constexpr (REG) {
        number(s0, held);
    } else {
        for (int s = s0; s < s1; s += 64) number(s, s + lane < s1 ? ids[s + lane] : -1);   // uniform in the wave
    }
}

static int bits_of(int E) {
    int b = 0;
    while ((1 << b) < E) ++b;
    return b;
}

static void launch_sort(const int* ids, int T, int E, int* offsets, int* row_of_slot, void* ws, hipStream_t st) {
    int* hist = static_cast<int*>(ws);
    const int bytes = place_words(E) * (int)sizeof(int);
    const int seg = sort_seg(T);
    auto place = [&](auto reg) {
        constexpr bool REG = decltype(reg)::value;
        static std::atomic<uint64_t> lds_set{0};
        if (bytes > 60 * 1024)                   // with the static words, over the default limit of 64 KiB
            allow_dynamic_lds(reinterpret_cast<const void*>(&moe_place_kernel<REG>),
                              place_words(kGroupedMaxExperts) * (int)sizeof(int), lds_set);
        hipLaunchKernelGGL(moe_place_kernel<REG>, dim3((T + seg - 1) / seg), dim3(SORT_NT), bytes, st, ids, T, E,
                           bits_of(E), seg, hist, offsets, row_of_slot);
    };
    hipLaunchKernelGGL(moe_count_kernel, dim3((T + seg - 1) / seg), dim3(SORT_NT), E * sizeof(int), st, ids, T, E, seg,
                       hist);
    if (seg == SORT_NT) place(std::true_type{});
    else place(std::false_type{});
}

// offsets of a call without slots
__global__ void moe_no_rows_kernel(int E, int* __restrict__ offsets) {
    for (int e = threadIdx.x; e <= E; e += 256) offsets[e] = 0;
}

// ---------------------------------------------------------------------------
// Token kernels.  A row is `chunks` pieces; `tpb` tokens share a workgroup when
// rows are short (tpb * span = 256 threads, span a power of two), else `parts`
// workgroups share a token, 256 pieces each.
// ---------------------------------------------------------------------------
struct TokenGrid {
    int span_log2;               // threads per token
    int parts;                   // workgroups per token
    unsigned blocks;
};

static TokenGrid token_grid(int B, int chunks) {
    TokenGrid g{};
    if (chunks >= 256) {
        g.span_log2 = 8;
        g.parts = (chunks + 255) / 256;
        g.blocks = (unsigned)B * (unsigned)g.parts;
    } else {
        while ((1 << g.span_log2) < chunks) ++g.span_log2;
        const int tpb = 256 >> g.span_log2;
        g.parts = 1;
        g.blocks = (unsigned)((B + tpb - 1) / tpb);
    }
    return g;
}

// token and piece of this thread; false: none
__device__ __forceinline__ bool token_piece(int B, int chunks, int span_log2, int parts, int& b, int& c) {
    if (parts > 1) {
        b = blockIdx.x / parts;
        c = (int)(blockIdx.x - b * parts) * 256 + (int)threadIdx.x;
    } else {
        b = (int)(blockIdx.x << (8 - span_log2)) + ((int)threadIdx.x >> span_log2);
        c = threadIdx.x & ((1 << span_log2) - 1);
    }
    return b < B && c < chunks;
}

// Slots of a token handled together: their row numbers, weights and rows are
// requested before the first is used.
constexpr int SLOTS = 8;

template <class V>
__global__ __launch_bounds__(256) void moe_gather_kernel(const V* __restrict__ rows, const float* __restrict__ scale,
                                                         const int* __restrict__ row_of_slot, int B, int k, int chunks,
                                                         int span_log2, int parts, V* __restrict__ out,
                                                         float* __restrict__ scale_out) {
    int b, c;
    if (!token_piece(B, chunks, span_log2, parts, b, c)) return;
    const int T = B * k;
    const V v = rows[(size_t)b * chunks + c];
    const float s = scale && c == 0 ? scale[b] : 0.0f;
    for (int j0 = 0; j0 < k; j0 += SLOTS) {
        int r[SLOTS];
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) r[j] = j0 + j < k ? row_of_slot[b * k + j0 + j] : -1;
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
            if ((unsigned)r[j] >= (unsigned)T) continue;
            out[(size_t)r[j] * chunks + c] = v;
            if (scale && c == 0) scale_out[r[j]] = s;
        }
    }
}

void launch_moe_gather(const void* rows, const float* scale, const int* row_of_slot, int B, int k, int row_bytes,
                       void* out, float* scale_out, hipStream_t st) {
    auto go = [&](auto* piece) {
        using V = std::remove_pointer_t<decltype(piece)>;
        const int chunks = row_bytes / (int)sizeof(V);
        const TokenGrid g = token_grid(B, chunks);
        hipLaunchKernelGGL(moe_gather_kernel<V>, dim3(g.blocks), dim3(256), 0, st, static_cast<const V*>(rows), scale,
                           row_of_slot, B, k, chunks, g.span_log2, g.parts, static_cast<V*>(out), scale_out);
    };
    if (row_bytes % 16 == 0) go((u32x4*)nullptr);
    else go((uint2*)nullptr);
}

// ---------------------------------------------------------------------------
// Few slots: sort and copy in one launch without a workspace.  The row of a slot
// is the number of slots before it in (expert, slot) order, so each token's
// workgroups count that over all T ids for their k slots (a ballot per 64 ids and
// slot) while the token's row is on its way from memory; one more workgroup
// writes the offsets.  The work grows with the workgroups times T: DIRECT_MAX_WORK
// bounds it (top-8 of 128, e4m3 rows of 2048, this / the two-launch sort and the
// copy, us: 192 tokens 6.2 / 8.4, 256 7.0 / 8.6, 512 10.6 / 9.7; top-2 of 8, rows of
// 4096: 512 5.0 / 7.9, 1024 8.5 / 9.5).
// ---------------------------------------------------------------------------
#ifndef QG_MOE_DIRECT_MAX_WORK
#define QG_MOE_DIRECT_MAX_WORK (5 << 18)
#endif

// work of `parts` workgroups per token
static int64_t direct_work(int B, int k, int parts) {
    return (int64_t)B * parts * ((k + SLOTS - 1) / SLOTS) * B * k;
}
static bool direct_sort(int B, int k) { return direct_work(B, k, 1) <= QG_MOE_DIRECT_MAX_WORK; }

template <class V>
__global__ __launch_bounds__(256) void moe_dispatch_direct_kernel(const int* __restrict__ ids, const V* __restrict__ rows,
                                                                  const float* __restrict__ scale, int B, int k, int E,
                                                                  int chunks, int parts, int* __restrict__ offsets,
                                                                  int* __restrict__ row_of_slot, V* __restrict__ out,
                                                                  float* __restrict__ scale_out) {
    const int T = B * k;
    const int tid = threadIdx.x;
    const int lane = tid & 63;
    const int wave = tid >> 6;
    if (blockIdx.x == gridDim.x - 1) {           // the offsets
        __shared__ int all[kGroupedMaxExperts];
        __shared__ int wave_total[4];
        for (int e = tid; e < E; e += 256) all[e] = 0;
        __syncthreads();
        for (int s = tid; s < T; s += 256) {
            const int e = ids[s];
            if (e >= 0 && e < E) atomicAdd(&all[e], 1);
        }
        __syncthreads();
        scan_experts<4>(all, E, nullptr, offsets, wave_total);
        return;
    }
    __shared__ int below[2][4][SLOTS];
    const int b = blockIdx.x / parts;
    const int part = blockIdx.x - b * parts;
    const int c = part * 256 + tid;
    V v{};
    if (c < chunks) v = rows[(size_t)b * chunks + c];
    const float s = scale && c == 0 ? scale[b] : 0.0f;
    for (int j0 = 0; j0 < k; j0 += SLOTS) {
        // (expert, slot) as one number: T <= DIRECT_MAX_WORK and E <= 2^10 fit 32 bits
        unsigned key[SLOTS];
        int n[SLOTS];
        unsigned kept = 0;                       // bit j: slot j has a row
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
            const int slot = b * k + j0 + j;
            const int e = j0 + j < k ? ids[slot] : -1;
            const bool in = e >= 0 && e < E;
            key[j] = in ? (unsigned)e * (unsigned)T + (unsigned)slot : 0u;
            kept |= in ? 1u << j : 0u;
            n[j] = 0;
        }
        for (int t0 = wave * 64; t0 < T; t0 += 256) {
            const int t = t0 + lane;
            const int e = t < T ? ids[t] : -1;
            const unsigned other = e >= 0 && e < E ? (unsigned)e * (unsigned)T + (unsigned)t : ~0u;
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) n[j] += __popcll(__ballot(other < key[j]));
        }
        int (*mine)[SLOTS] = below[(j0 / SLOTS) & 1];
        if (lane == 0) {
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) mine[wave][j] = n[j];
        }
        __syncthreads();                         // the other half of `below` is free again after it
        int r[SLOTS];
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) r[j] = mine[0][j] + mine[1][j] + mine[2][j] + mine[3][j];
        if (c < chunks) {
#pragma unroll
            for (int j = 0; j < SLOTS; ++j)
                if (kept >> j & 1) out[(size_t)r[j] * chunks + c] = v;
        }
        if (c == 0) {
#pragma unroll
            for (int j = 0; j < SLOTS; ++j) {
                if (j0 + j < k) row_of_slot[b * k + j0 + j] = kept >> j & 1 ? r[j] : -1;
                if (scale && (kept >> j & 1)) scale_out[r[j]] = s;
            }
        }
    }
}

size_t moe_dispatch_workspace_bytes(int B, int k, int E) {
    if (B == 0 || direct_sort(B, k)) return 0;
    const int T = B * k;
    const int seg = sort_seg(T);
    return (size_t)((T + seg - 1) / seg) * E * sizeof(int);
}

void launch_moe_dispatch(const int* ids, const void* rows, const float* scale, int B, int k, int E, int row_bytes,
                         int* offsets, int* row_of_slot, void* out, float* scale_out, void* ws, hipStream_t st) {
    if (B == 0) {
        hipLaunchKernelGGL(moe_no_rows_kernel, dim3(1), dim3(256), 0, st, E, offsets);
        return;
    }
    if (direct_sort(B, k)) {
        auto go = [&](auto* piece, const void* in, int chunks, int parts) {
            using V = std::remove_pointer_t<decltype(piece)>;
            hipLaunchKernelGGL(moe_dispatch_direct_kernel<V>, dim3((unsigned)(B * parts + 1)), dim3(256), 0, st, ids,
                               static_cast<const V*>(in), in ? scale : nullptr, B, k, E, chunks, parts, offsets,
                               row_of_slot, static_cast<V*>(out), scale_out);
        };
        const int piece = row_bytes % 16 == 0 ? 16 : 8;
        const int chunks = rows ? row_bytes / piece : 0;
        const int parts = std::max(1, (chunks + 255) / 256);
        // every part of a long row would count again: sort first, then copy
        if (parts > 1 && direct_work(B, k, parts) > QG_MOE_DIRECT_MAX_WORK) {
            go((u32x4*)nullptr, nullptr, 0, 1);
            launch_moe_gather(rows, scale, row_of_slot, B, k, row_bytes, out, scale_out, st);
        } else if (piece == 16) {
            go((u32x4*)nullptr, rows, chunks, parts);
        } else {
            go((uint2*)nullptr, rows, chunks, parts);
        }
        return;
    }
    launch_sort(ids, B * k, E, offsets, row_of_slot, ws, st);
    if (rows) launch_moe_gather(rows, scale, row_of_slot, B, k, row_bytes, out, scale_out, st);
}

// STREAM: the experts' rows, dead after this, pass the caches by (8192 tokens of
// top-8, 2048 bf16, 65 us without, 60 with; 4096 of top-2, 4096 bf16, 26.7 and 24.8).
template <bool STREAM>
__global__ __launch_bounds__(256) void moe_combine_kernel(const u32x4* __restrict__ rows,
                                                          const int* __restrict__ row_of_slot,
                                                          const float* __restrict__ weights, const u32x4* residual, int B,
                                                          int k, int chunks, int span_log2, int parts, u32x4* y) {
    int b, c;
    if (!token_piece(B, chunks, span_log2, parts, b, c)) return;
    const int T = B * k;
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.0f;
    const size_t at = (size_t)b * chunks + c;
    u32x4 res{0u, 0u, 0u, 0u};
    if (residual) res = residual[at];
    for (int j0 = 0; j0 < k; j0 += SLOTS) {
        int r[SLOTS];
        float w[SLOTS];
        u32x4 v[SLOTS];
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
            const bool in = j0 + j < k;
            r[j] = in ? row_of_slot[b * k + j0 + j] : -1;
            w[j] = in && weights ? weights[b * k + j0 + j] : 1.0f;
        }
#pragma unroll
        for (int j = 0; j < SLOTS; ++j)
            if ((unsigned)r[j] < (unsigned)T) v[j] = load_row<STREAM>(rows + (size_t)r[j] * chunks + c);
#pragma unroll
        for (int j = 0; j < SLOTS; ++j) {
            if ((unsigned)r[j] >= (unsigned)T) continue;
            float f[8];
            unpack8(v[j], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) acc[i] = fmaf(w[j], f[i], acc[i]);
        }
    }
    if (residual) {
        float v[8];
        unpack8(res, v);
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += v[i];
    }
    y[at] = pack8(acc);
}

void launch_moe_combine(const uint16_t* rows, const int* row_of_slot, const float* weights, const uint16_t* residual,
                        int B, int k, int K, uint16_t* y, hipStream_t st) {
    const int chunks = K / 8;
    const TokenGrid g = token_grid(B, chunks);
    auto go = [&](auto stream) {
        hipLaunchKernelGGL(moe_combine_kernel<decltype(stream)::value>, dim3(g.blocks), dim3(256), 0, st,
                           reinterpret_cast<const u32x4*>(rows), row_of_slot, weights,
                           reinterpret_cast<const u32x4*>(residual), B, k, chunks, g.span_log2, g.parts,
                           reinterpret_cast<u32x4*>(y));
    };
    if ((size_t)B * k * K * 2 > kStreamBytes) go(std::true_type{});
    else go(std::false_type{});
}

// NT threads per token, a workgroup or (rows of up to 64 pieces) a wave: 16384 tokens
// of top-4, 128 / 512 bf16, 12.0 / 30.5 us with a wave, 21.6 / 33.4 with a workgroup.
// They hold the pieces of dy, and the slots' products <dy, row> are reduced over
// them, J slots and SLOTS / J pieces a thread at a time (J = 2, 4 or 8, the least
// that covers k: with 8 alone, 4096 tokens of top-2, 4096 bf16, took 37 us, so 34).
// drows passes the caches by, which then keep the rows (4099 / 1000 / 256 tokens of
// top-8, 2048 bf16, 59 / 18.1 / 6.3 us without, 57 / 15.8 / 5.7 with).
#ifndef QG_MOE_BWD_WAVE_K          // longest row of one wave per token
#define QG_MOE_BWD_WAVE_K 512
#endif
template <int NT, int J>
__global__ __launch_bounds__(256) void moe_combine_backward_kernel(
    const u32x4* __restrict__ dy, const u32x4* __restrict__ rows, const int* __restrict__ row_of_slot,
    const float* __restrict__ weights, int B, int k, int chunks, u32x4* __restrict__ drows, float* __restrict__ dweights) {
    constexpr int U = SLOTS / J;
    __shared__ float red[4][J];
    const int b = NT == 64 ? (int)(blockIdx.x * 4 + (threadIdx.x >> 6)) : (int)blockIdx.x;
    if (b >= B) return;                          // whole waves, where no barrier follows
    const int T = B * k;
    const int tid = threadIdx.x % NT;
    for (int j0 = 0; j0 < k; j0 += J) {
        int r[J];
        float w[J], dot[J];
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const bool in = j0 + j < k;
            r[j] = in ? row_of_slot[b * k + j0 + j] : -1;
            if ((unsigned)r[j] >= (unsigned)T) r[j] = -1;
            w[j] = in && weights ? weights[b * k + j0 + j] : 1.0f;
            dot[j] = 0.0f;
        }
        for (int c0 = tid; c0 < chunks; c0 += NT * U) {
            u32x4 d[U], v[U][J];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * NT;
                if (c >= chunks) continue;
                d[u] = dy[(size_t)b * chunks + c];
                if (dweights) {
#pragma unroll
                    for (int j = 0; j < J; ++j)
                        if (r[j] >= 0) v[u][j] = rows[(size_t)r[j] * chunks + c];
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int c = c0 + u * NT;
                if (c >= chunks) continue;
                float g[8];
                unpack8(d[u], g);
#pragma unroll
                for (int j = 0; j < J; ++j) {
                    if (r[j] < 0) continue;
                    float f[8];
                    if (drows) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) f[i] = w[j] * g[i];
                        store_row<true>(drows + (size_t)r[j] * chunks + c, pack8(f));
                    }
                    if (dweights) {
                        unpack8(v[u][j], f);
#pragma unroll
                        for (int i = 0; i < 8; ++i) dot[j] = fmaf(g[i], f[i], dot[j]);
                    }
                }
            }
        }
        if (dweights) {
#pragma unroll
            for (int j = 0; j < J; ++j) {
                dot[j] = wave_sum(dot[j]);
                if (NT == 64 && tid == 0 && j0 + j < k) dweights[b * k + j0 + j] = dot[j];
                if (NT > 64 && (tid & 63) == 0) red[tid >> 6][j] = dot[j];
            }
            if constexpr (NT > 64) {
                __syncthreads();
                if (tid < J && j0 + tid < k)
                    dweights[b * k + j0 + tid] = red[0][tid] + red[1][tid] + red[2][tid] + red[3][tid];
                __syncthreads();
            }
        }
    }
}

void launch_moe_combine_backward(const uint16_t* dy, const uint16_t* rows, const int* row_of_slot, const float* weights,
                                 int B, int k, int K, uint16_t* drows, float* dweights, hipStream_t st) {
    auto go = [&](auto nt, auto j) {
        constexpr int NT = decltype(nt)::value;
        hipLaunchKernelGGL((moe_combine_backward_kernel<NT, decltype(j)::value>), dim3(NT == 64 ? (B + 3) / 4 : B), dim3(256),
                           0, st, reinterpret_cast<const u32x4*>(dy), reinterpret_cast<const u32x4*>(rows), row_of_slot,
                           weights, B, k, K / 8, reinterpret_cast<u32x4*>(drows), dweights);
    };
    auto by_row = [&](auto j) {
        if (K <= QG_MOE_BWD_WAVE_K) go(ic<64>{}, j);
        else go(ic<256>{}, j);
    };
    if (k <= 2) by_row(ic<2>{});
    else if (k <= 4) by_row(ic<4>{});
    else by_row(ic<8>{});
}

}  // namespace qg
