// Causal attention of a batch's new tokens over their paged cache.
//
//   out[t, h] = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale q . k_j - max_j)
//   j over the positions up to the token's own; with a window W those less than W before
//   it and the first `sinks` positions of the sequence
//
// One pass over the keys with a running maximum m and sum l in fp32 (base-2
// exponentials).  Scores are formed transposed, S^T = K Q^T, so that a lane of the
// matrix instruction's result holds one query's scores: the row statistics of the
// softmax need no LDS, the factors that rescale the running result are the lane's own,
// and the probabilities are, without a move, the second operand of O^T = V^T P^T (the
// order of the keys inside a step is free as long as both operands share it).  Its
// first operand is read transposed from LDS (ds_read_b64_tr).  The rows of a matrix tile are
// (token, query head of the group) pairs of one key head: a key is read once for its
// whole group.
//
// What a masked key holds never matters: its probability is an exact zero, values that
// no row sees are replaced by zeros before the product (uninitialised memory may hold
// NaN), and a step with a value that only some rows see and that is infinite or NaN is
// multiplied apart, row by row or key by key.  A row that sees no key is zero, its lse
// minus infinity.

#include <algorithm>
#include <atomic>

#include "device_common.h"
#include "formats.h"
#include "launch.h"
#include "rows.h"
#include "sequences.h"

namespace qg {

namespace {

// ---------------------------------------------------------------------------
// What both kernels share: the call, its keys, its work items.
// ---------------------------------------------------------------------------
struct Call : AttentionArgs {
    int G;                       // query heads of a key head
    float scale2;                // scale log2(e)
    // the plan
    int items;                   // work items for each key head at most, below 2^24
    int few, few_rows;           // few = 1: sequences of up to few_rows rows; 0: the others; -1: all
    int target;                  // chunks wanted for each key head over the whole batch; 0: keys are not split
    int least;                   // tiles of a chunk at least
    unsigned* counters;          // one a split row tile, zero between calls
    float* slots;                // partial results of chunks
    bool stream;                 // the cache is read once, past the caches
    int shared;                  // positions below are found by row 0 of the table
    // partial results of the shared prefix: [chunks, Hkv, T G] rows of D elements, (m, l) each
    int prior_chunks;
    float *prior, *prior_ml;
};

// Key tiles that some token of a sequence sees: [begin0, end0) around the first
// positions and [begin1, end1), in tiles of TK positions.
struct Span {
    int begin0, begin1, n0, n;
    __device__ __forceinline__ int tile(int i) const { return i < n0 ? begin0 + i : begin1 + i - n0; }
};
template <int TK>
__device__ __forceinline__ Span span_of(const Call& a, const Sequence& s) {
    const int limit = (int)min((int64_t)s.len, (int64_t)a.max_pages << a.page_shift);
    int lo = a.prefix, seen_first = 0;
    if (a.window > 0) {
        lo = max(lo, min(s.len - s.tokens - a.window + 1, limit));       // (a length past the table leaves no tile)
        seen_first = min(min(a.sinks, lo), limit);
    }
    Span r;
    r.begin1 = lo / TK;
    const int end1 = max((limit + TK - 1) / TK, r.begin1);
    r.begin0 = a.prefix / TK;
    r.n0 = seen_first > a.prefix ? min((seen_first + TK - 1) / TK, r.begin1) - r.begin0 : 0;
    r.n = r.n0 + end1 - r.begin1;
    return r;
}

// A work item: a tile of at most BM rows of a sequence and a chunk of the key tiles.
struct Item {
    int b, row0, chunk, chunks, chunk_tiles, first;      // first: the item of the row tile's first chunk
    Sequence s;
    Span span;
};

// The items are numbered sequence by sequence, row tile by row tile, chunk by chunk.  A
// chunk's length follows from the whole batch: total / target tiles, so that chunks are alike
// whatever the lengths, and there are at most target + (row tiles) of them.  Every wave
// finds the item `it` for itself, 64 sequences a step, on scans of DPP moves (false: there
// is none).  BY_TILE: `it` numbers the row tiles, the item is the tile's first chunk.
template <int BM, int TK, bool LAST_FIRST, bool BY_TILE = false>
__device__ __forceinline__ bool find_item(const Call& a, int it, Item& item) {
    const int lane = threadIdx.x & 63;
    const int blocks = (a.B + 63) >> 6;
    auto load = [&](int j, int& lo, int& hi, int& len) {
        const int b = 64 * j + lane;
        lo = a.q_offsets[min(b, a.B)];
        hi = a.q_offsets[min(b + 1, a.B)];
        len = a.kv_len[min(b, a.B - 1)];
    };
    auto rows_of = [&](const Sequence& s) {
        const int rows = s.tokens * a.G;
        return a.few < 0 || (rows <= a.few_rows) == (a.few != 0) ? (rows + BM - 1) / BM : 0;
    };
    int chunk_tiles = 0x7fffffff;
    int lo, hi, len;
    load(0, lo, hi, len);
    if (a.target > 0) {
        double total = 0.0;                              // exact: below 2^53
        int l = lo, h = hi, k = len;
        for (int j = 0; j < blocks; ++j) {
            const Sequence s = sequence_of(l, h, k, a.T);
            if (j + 1 < blocks) load(j + 1, l, h, k);
            if (64 * j + lane < a.B) total += (double)rows_of(s) * (double)span_of<TK>(a, s).n;
        }
        total = wave_sum(total);
        chunk_tiles = max(a.least, (int)fmin(ceil(total / a.target), 2147483647.0));
    }
    int carry = 0, carry_items = 0;
    for (int j = 0; j < blocks; ++j) {
        const int b = 64 * j + lane;
        const Sequence s = sequence_of(lo, hi, len, a.T);
        if (j + 1 < blocks) load(j + 1, lo, hi, len);
        const int rows = b < a.B ? rows_of(s) : 0;
        const int n = span_of<TK>(a, s).n;
        const int chunks = a.target > 0 ? max(1, (n - 1) / chunk_tiles + 1) : 1;
        // (a count past the grid is as good as any other: sums stay inside an int)
        const int items = (int)min((int64_t)rows * chunks, (int64_t)1 << 24);
        const int count = BY_TILE ? rows : items;
        const int incl = wave_scan(count) + carry;
        const int incl_items = BY_TILE ? wave_scan(items) + carry_items : incl;
        const int total = __builtin_amdgcn_readlane(incl, 63);
        if (it < total) {
            const int before = incl - count;
            const int src = __builtin_ctzll(__ballot(it >= before && it < incl));
            item.b = __builtin_amdgcn_readfirstlane(64 * j + src);
            item.s.first_token = __builtin_amdgcn_readlane(s.first_token, src);
            item.s.tokens = __builtin_amdgcn_readlane(s.tokens, src);
            item.s.len = __builtin_amdgcn_readlane(s.len, src);
            item.chunks = __builtin_amdgcn_readlane(chunks, src);
            const int at = it - __builtin_amdgcn_readlane(before, src);
            const int tile = BY_TILE ? at : at / item.chunks;
            // the last rows of a sequence see the most keys: their tiles begin first
            item.row0 = (LAST_FIRST ? __builtin_amdgcn_readlane(rows, src) - 1 - tile : tile) * BM;
            item.chunk = BY_TILE ? 0 : at % item.chunks;
            item.first = BY_TILE ? __builtin_amdgcn_readlane(incl_items - items, src) + tile * item.chunks : it - item.chunk;
            item.span = span_of<TK>(a, item.s);
            item.chunk_tiles = (item.span.n + item.chunks - 1) / item.chunks;
            // offsets that do not ascend may ask for more than the grid holds: such a tile is left out whole
            return item.first + item.chunks <= a.items;
        }
        carry = total;
        if (BY_TILE) carry_items = min(__builtin_amdgcn_readlane(incl_items, 63), 1 << 24);
    }
    return false;
}

// The larger of the two lanes' values at distance 16 / 32, and their sum, in both.
__device__ __forceinline__ float both16(float v, float& other) {
    const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    other = __uint_as_float(r[1]);
    return __uint_as_float(r[0]);
}
__device__ __forceinline__ float both32(float v, float& other) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
    other = __uint_as_float(r[1]);
    return __uint_as_float(r[0]);
}

// 16 bytes a lane from base + off to lds + 16 lane, as lds_copy_b128 of device_common.h.
__device__ __forceinline__ void lds_copy_b128(const void* base, uint32_t off, uint32_t lds) {
    asm volatile("global_load_lds_dwordx4 %0, %1" : : "v"(off), "s"(base), "{m0}"(lds) : "memory");
}
// The same past the caches (bytes that nothing reads again soon).
__device__ __forceinline__ void lds_copy_b128_nt(const void* base, uint32_t off, uint32_t lds) {
    asm volatile("global_load_lds_dwordx4 %0, %1 nt" : : "v"(off), "s"(base), "{m0}"(lds) : "memory");
}
// 4 bytes a lane from src to lds + 4 lane
__device__ __forceinline__ void lds_copy_b32(const void* src, uint32_t lds) {
    asm volatile("global_load_lds_dword %0, off" : : "v"(src), "{m0}"(lds) : "memory");
}
template <int N>
__device__ __forceinline__ void wait_vmem() {
    asm volatile("s_waitcnt vmcnt(%0)" : : "n"(N) : "memory");
}

// Waits for all but the copies of the tiles behind this one: `left` remain, at most MOST have
// been requested.
template <int COPIES, int MOST>
__device__ __forceinline__ void wait_tiles(int left) {
    if (left >= MOST) wait_vmem<MOST * COPIES>();
    else if (MOST > 1 && left == MOST - 1) wait_vmem<(MOST > 1 ? MOST - 1 : 0) * COPIES>();
    else if (MOST > 2 && left == MOST - 2) wait_vmem<(MOST > 2 ? MOST - 2 : 0) * COPIES>();
    else wait_vmem<0>();
}
// Waits for all but the copies behind what is needed: `first` of them, and TILE for each of
// the tiles that follow in LDS (`left` remain, at most NS - 1 are there).
template <int NS, int TILE, int FIRST>
__device__ __forceinline__ void wait_behind(int left, bool first = true) {
    if (first) {
        if (left >= NS - 1) wait_vmem<(NS - 1) * TILE + FIRST>();
        else if (NS > 2 && left == NS - 2) wait_vmem<(NS > 2 ? NS - 2 : 0) * TILE + FIRST>();
        else if (NS > 3 && left == NS - 3) wait_vmem<(NS > 3 ? NS - 3 : 0) * TILE + FIRST>();
        else wait_vmem<FIRST>();
    } else {
        if (NS > 1 && left >= NS - 1) wait_vmem<(NS - 1) * TILE>();
        else if (NS > 2 && left == NS - 2) wait_vmem<(NS > 2 ? NS - 2 : 0) * TILE>();
        else if (NS > 3 && left == NS - 3) wait_vmem<(NS > 3 ? NS - 3 : 0) * TILE>();
        else wait_vmem<0>();
    }
}

typedef short i16x4 __attribute__((ext_vector_type(4)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Transposed LDS reads: the 16 lanes of a group name 8-byte pieces that make the rows
// of a matrix 16 columns wide (bf16: 4 lanes a row, e4m3: 2), and lane i receives column i.
__device__ __forceinline__ u32x2 lds_columns_b16(uint32_t at) {
    const auto p = (__attribute__((address_space(3))) i16x4*)(uintptr_t)at;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr16_b64_v4i16(p));
}
__device__ __forceinline__ u32x2 lds_columns_b8(uint32_t at) {
    const auto p = (__attribute__((address_space(3))) i32x2*)(uintptr_t)at;
    return __builtin_bit_cast(u32x2, __builtin_amdgcn_ds_read_tr8_b64_v2i32(p));
}
template <class T>
__device__ __forceinline__ void lds_write(uint32_t at, T v) {
    *(__attribute__((address_space(3))) T*)(uintptr_t)at = v;
}
template <class T>
__device__ __forceinline__ T lds_read(uint32_t at) {
    return *(const __attribute__((address_space(3))) T*)(uintptr_t)at;
}

// Eight e4m3 codes as bf16: exact.
__device__ __forceinline__ u32x4 e4m3_to_bf16(u32x2 c) {
    u32x4 r;
    r.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.x, 1.0f, false));
    r.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.x, 1.0f, true));
    r.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.y, 1.0f, false));
    r.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c.y, 1.0f, true));
    return r;
}

// An entry of a list that is the same for the whole wave and does not change under the
// launch: a scalar load, which waits for no copy in flight (as a vector load it would
// share their counter, and wait for all of them).
__device__ __forceinline__ int load_scalar(const int* p) {
    return *(const __attribute__((address_space(4))) int*)(uintptr_t)p;
}

// Ends the compiler's wait for loaded registers here.  It does not know the copies to LDS:
// a register still awaited in the loop would make every tile wait for the copies behind it.
template <int N>
__device__ __forceinline__ void arrived(bf16x8 (&q)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+v"(q[i]));
}

// Keeps an array in memory, out of the registers.
template <class T>
__device__ __forceinline__ void in_memory(T& array) {
    asm volatile("" : : "v"(&array) : "memory");
}

// Bits 0 .. n: none for a negative n, all from 63 on.
__device__ __forceinline__ uint64_t bits_to(int n) {
    return n < 0 ? 0ull : ~0ull >> (63 - min(n, 63));
}

// An infinity or NaN among eight bf16 values.
__device__ __forceinline__ bool nonfinite8(u32x4 v) {
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t w = v[i];
        bad |= (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
    }
    return bad;
}

// ---- the running softmax of one query column -------------------------------------
// m: what is subtracted from the column's scores (base 2), the same in all its lanes; l:
// this lane's share of the sum.  m follows the largest score only when that has grown by
// more than kSlack: exponentials up to 2^kSlack cost fp32 sums and bf16 probabilities
// nothing, and the running result is rarely rescaled after its first tile.
constexpr float kSlack = 8.0f;
// The larger score; a NaN stays one (its row is NaN whatever is subtracted), which spares
// the instructions that would quiet it.
__device__ __forceinline__ float larger(float a, float b) { return __builtin_elementwise_maximum(a, b); }
struct Running {
    float m = -__builtin_inff(), l = 0.0f;
    // The reference to subtract: a column that has seen nothing keeps its exponentials at zero.
    __device__ __forceinline__ float reference() const { return m == -__builtin_inff() ? 0.0f : m; }
    // whether a tile's largest score moves the reference
    __device__ __forceinline__ bool outgrown(float top) const { return top > m + kSlack; }
    // moves it in the lanes that need it; the factor of what was summed before
    __device__ __forceinline__ float follow(float top) {
        const float before = m;
        if (outgrown(top)) m = top;
        const float w = __builtin_amdgcn_exp2f(before - reference());
        l *= w;
        return w;
    }
};

// Joins the partial results of a row's chunks, in order: `o` of N elements with (m, l).
template <int N>
struct Joined {
    float m = -__builtin_inff(), l = 0.0f, o[N];
    __device__ __forceinline__ Joined() {
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = 0.0f;
    }
    __device__ __forceinline__ void add(float m2, float l2, const float* o2) {
        const float top = fmaxf(m, m2);
        const float ref = top == -__builtin_inff() ? 0.0f : top;
        const float w1 = __builtin_amdgcn_exp2f(m - ref), w2 = __builtin_amdgcn_exp2f(m2 - ref);
        m = top;
        l = l * w1 + l2 * w2;
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] = o[i] * w1 + o2[i] * w2;
    }
};

// Agent-scope accesses of N floats, two at a time: other XCDs read what this one wrote.
template <int N>
__device__ __forceinline__ void store_agent(float* p, const float* v) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const uint64_t u = (uint64_t)__float_as_uint(v[i]) | ((uint64_t)__float_as_uint(v[i + 1]) << 32);
        __hip_atomic_store(reinterpret_cast<uint64_t*>(p + i), u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
}
template <int N>
__device__ __forceinline__ void load_agent(const float* p, float* v) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
        const uint64_t u = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p + i), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        v[i] = __uint_as_float((uint32_t)u);
        v[i + 1] = __uint_as_float((uint32_t)(u >> 32));
    }
}

// N elements of a row's result, rounded, and its lse.
template <int N>
__device__ __forceinline__ void rounded(const Joined<N>& j, uint32_t (&w)[N / 2]) {
    const float inv = 1.0f / j.l;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const f32x2 v = j.l == 0.0f ? f32x2{0.0f, 0.0f} : f32x2{j.o[2 * i] * inv, j.o[2 * i + 1] * inv};
        w[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(v, bf16x2));
    }
}
__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.0f ? -__builtin_inff() : (m + log2f(l)) * 0.69314718055994530942f;
}

// A row's result: N neighbouring elements from element d0, and once a row the lse.
template <int N>
__device__ __forceinline__ void store_row(const Call& a, int D, int64_t row, int d0, const Joined<N>& j) {
    uint32_t w[N / 2];
    rounded<N>(j, w);
    uint16_t* p = a.out + row * D + d0;
    if constexpr (N == 8) *reinterpret_cast<u32x4*>(p) = u32x4{w[0], w[1], w[2], w[3]};
    else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    if (a.lse && d0 == 0) a.lse[row] = lse_of(j.m, j.l);
}

// ---------------------------------------------------------------------------
// Few rows a sequence (decoding): a workgroup takes one row tile of 16 and a chunk of
// keys, its four waves 32 keys each of every 128.  Every wave streams its keys and
// values through buffers of its own in LDS, with no barrier until its end: a buffer is
// requested again as soon as its product has read it, so keys arrive under a tile's softmax
// and second product and values under the next one's first.  The waves' results
// are joined in LDS, those of chunks by the last workgroup to arrive, in chunk order.
//
// Bound by memory: two workgroups a CU keep 100 KB on their way.  64 sequences of 8192 keys
// take 330 us (6.5 TB/s), of ragged lengths in e4m3 120 (5.5); one of 16384 20.4 (3.3), 7 of
// them latency before and behind the stream.  The probabilities
// enter the second product as a sum of two bf16 numbers, so it loses nothing to their
// rounding (matrix instructions are idle here).
// ---------------------------------------------------------------------------
template <int D, bool E4M3>
struct Rows {
    static constexpr int BM = 16, TK = 32, WAVES = 4, TILE = TK * WAVES;
    static constexpr int RB = E4M3 ? D : 2 * D;          // bytes of a cached row
    static constexpr int PIECES = RB / 16;
    static constexpr int KEYS = 64 / PIECES;             // keys of one copy
    static constexpr int LOADS = TK / KEYS;
    static constexpr int NS = 256 / RB;                  // tiles in LDS for each wave
    static constexpr int KCOPIES = LOADS + (E4M3 ? 1 : 0), VCOPIES = LOADS;      // of a tile; scales come with the keys
    static constexpr int K0 = 0, V0 = TK * RB, S0 = 2 * TK * RB, STAGE = S0 + (E4M3 ? 256 : 0);
    static constexpr int WAVE_BYTES = NS * STAGE;
    static constexpr int LDS = WAVES * WAVE_BYTES + 16;
    static constexpr int OROW = D + 4;                   // floats of a row handed over in LDS
    static constexpr int SLOT = BM * (D + 2);            // floats
    static_assert(BM * (OROW + 2) * 4 <= WAVE_BYTES && 256 * (16 * 8 + D / 16 * 4) <= WAVES * WAVE_BYTES, "LDS");
    // Where a row's 16-byte piece lies: pieces change places by the key so that the lanes
    // of a read meet different banks (16 pieces span all of them).
    __device__ static __forceinline__ int swap_k(int key) {
        return PIECES == 16 ? key & 15 : PIECES == 8 ? (key >> 1) & 7 : (key >> 2) & 3;
    }
    __device__ static __forceinline__ int swap_v(int key) {
        if (!E4M3) return PIECES == 16 ? (key & 3) * 4 + (key >> 2 & 1) * 2 : (key >> 1 & 1) * 2 + (key >> 2 & 1) * 4;
        return PIECES == 8 ? (key >> 1 & 1) + (key >> 4 & 1) * 2 + (key >> 2 & 1) * 4 : (key >> 4 & 1) + (key >> 2 & 1) * 2;
    }
};

// The larger value, and the sum, of 16 neighbouring lanes, in each of them.
__device__ __forceinline__ float max_of_16(float v) {
    v = fmaxf(v, dpp<0xb1>(v));
    v = fmaxf(v, dpp<0x4e>(v));
    v = fmaxf(v, dpp<0x141>(v));
    return fmaxf(v, dpp<0x140>(v));
}
__device__ __forceinline__ float sum_of_16(float v) {
    v += dpp<0xb1>(v);
    v += dpp<0x4e>(v);
    v += dpp<0x141>(v);
    return v + dpp<0x140>(v);
}

// What the join of parts needs of a workgroup's LDS: the (m, l) of 16 rows of at most 256
// parts, and a sum from every thread.
constexpr int kParts = 256, kJoinSums = kParts * 16 * 8;
template <int D>
constexpr int kJoinBytes = kJoinSums + 256 * (D / 16) * 4;

// Joins all parts of up to 16 rows at once: `own` chunks in slots (`stride` floats apart, (m, l)
// of the rows from `ml_at` on), and those of a shared prefix (its rows from `row0` on).  First
// every part's (m, l), then its weight, then the weighted sums, the parts dealt to as many
// threads as there are: three trips to memory, whatever their number.  Thread t
// receives elements t % 16 * D / 16 .. of row t / 16 in j, which with no chunk of its own is
// one more part.
template <int D>
__device__ __forceinline__ void join_parts(const Call& a, unsigned char* smem, int h, int rows, int64_t row0, const float* slot,
                                           int64_t stride, int ml_at, int own, Joined<D / 16>& j) {
    constexpr int N = D / 16;
    const int tid = threadIdx.x, r = tid >> 4, d0 = (tid & 15) * N;
    const bool live = r < rows;
    const int parts = own + a.prior_chunks;
    const int64_t prior_rows = (int64_t)a.T * a.G;
    float* ml = reinterpret_cast<float*>(smem);
    __syncthreads();
    for (int x = tid; x < parts * 16; x += 256) {
        const int part = x / 16, pr = x % 16;
        if (pr >= rows) continue;
        if (part < own) load_agent<2>(slot + part * stride + ml_at + 2 * pr, ml + 2 * x);
        else
            *reinterpret_cast<f32x2*>(ml + 2 * x) =
                *reinterpret_cast<const f32x2*>(a.prior_ml + 2 * (((int64_t)(part - own) * a.Hkv + h) * prior_rows + row0 + pr));
    }
    __syncthreads();
    float m = own ? -__builtin_inff() : j.m, l = 0.0f;
    if (live) {
        for (int x = tid & 15; x < parts; x += 16) m = fmaxf(m, ml[2 * (x * 16 + r)]);
        m = max_of_16(m);
        const float ref = m == -__builtin_inff() ? 0.0f : m;
        for (int x = tid & 15; x < parts; x += 16) {
            float* at = ml + 2 * (x * 16 + r);
            const float w = __builtin_amdgcn_exp2f(at[0] - ref);
            l += at[1] * w;
            at[0] = w;
        }
        l = sum_of_16(l);
    }
    __syncthreads();
    const int sets = 16 / rows, set = r / rows, pr = r % rows;
    float sum[N];
#pragma unroll
    for (int e = 0; e < N; ++e) sum[e] = 0.0f;
    if (set < sets) {
#pragma unroll 4
        for (int x = set; x < own; x += sets) {
            float v[N];
            load_agent<N>(slot + x * stride + pr * D + d0, v);
            const float w = ml[2 * (x * 16 + pr)];
#pragma unroll
            for (int e = 0; e < N; ++e) sum[e] = fmaf(v[e], w, sum[e]);
        }
#pragma unroll 4
        for (int x = set; x < a.prior_chunks; x += sets) {
            const float* v = a.prior + (((int64_t)x * a.Hkv + h) * prior_rows + row0 + pr) * D + d0;
            const float w = ml[2 * ((own + x) * 16 + pr)];
#pragma unroll
            for (int e = 0; e < N; ++e) sum[e] = fmaf(v[e], w, sum[e]);
        }
    }
    float* sums = reinterpret_cast<float*>(smem + kJoinSums);
#pragma unroll
    for (int e = 0; e < N; ++e) sums[tid * N + e] = sum[e];
    __syncthreads();
    if (!live) return;
    for (int x = 1; x < sets; ++x)
#pragma unroll
        for (int e = 0; e < N; ++e) sum[e] += sums[(x * rows * 16 + tid) * N + e];
    const float w = own ? 0.0f : __builtin_amdgcn_exp2f(j.m - (m == -__builtin_inff() ? 0.0f : m));
#pragma unroll
    for (int e = 0; e < N; ++e) j.o[e] = own ? sum[e] : fmaf(j.o[e], w, sum[e]);
    j.l = own ? l : fmaf(j.l, w, l);
    j.m = m;
}

template <int D, bool E4M3>
__global__ __launch_bounds__(256, 2) void attention_rows_kernel(Call a) {
    using R = Rows<D, E4M3>;
    extern __shared__ __attribute__((aligned(256))) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 15, g = lane >> 4;              // column (row of the tile), lane group
    const int h = blockIdx.x % a.Hkv;
    Item item;
    if (!find_item<R::BM, R::TILE, false>(a, (int)(blockIdx.x / a.Hkv), item)) return;
    const int first_pos = item.s.len - item.s.tokens;
    const int rows = min(R::BM, item.s.tokens * a.G - item.row0);
    const int my_row = item.row0 + c;
    const bool mine = c < rows;
    const int pos = mine ? max(first_pos + my_row / a.G, -1) : -1;
    const int pos_min = first_pos + item.row0 / a.G, pos_max = first_pos + (item.row0 + rows - 1) / a.G;
    const int limit = (int)min((int64_t)item.s.len, (int64_t)a.max_pages << a.page_shift);

    const int i0 = item.chunk * item.chunk_tiles;        // (a last chunk may be left without tiles)
    const int tiles = min(item.chunk_tiles, item.span.n - i0);
    const uint32_t ring = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)smem + wave * R::WAVE_BYTES;

    // the copies' offsets from a 16-key half's first row
    uint32_t koff[R::LOADS], voff[R::LOADS];
#pragma unroll
    for (int j = 0; j < R::LOADS; ++j) {
        const int key = j * R::KEYS + lane / R::PIECES;
        const int at = (key & 15) * R::RB;
        koff[j] = at + ((lane % R::PIECES) ^ R::swap_k(key)) * 16;
        voff[j] = at + ((lane % R::PIECES) ^ R::swap_v(key)) * 16;
    }
    // the two pages of a wave's 32 keys: their rows in the cache, -1 where there is no page
    struct Pages { int64_t row[2]; };
    auto pages_of = [&](int key0) {
        Pages p;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int key = key0 + 16 * x;
            const int64_t b = key < a.shared ? 0 : item.b;
            const int id = key < limit ? load_scalar(a.table + b * a.max_pages + (key >> a.page_shift)) : -1;
            p.row[x] = id >= 0 && id < a.pages
                ? ((((int64_t)id * a.Hkv + h) << a.page_shift) + (key & ((1 << a.page_shift) - 1))) : -1;
        }
        return p;
    };
    auto key_of = [&](int i) { return item.span.tile(i0 + i) * R::TILE + wave * R::TK; };
    auto copy_rows = [&](const void* cache, const uint32_t (&off)[R::LOADS], uint32_t to, int64_t row0, int64_t row1) {
        const unsigned char* half0 = static_cast<const unsigned char*>(cache) + row0 * R::RB;
        const unsigned char* half1 = static_cast<const unsigned char*>(cache) + row1 * R::RB;
        if (a.stream) {
#pragma unroll
            for (int j = 0; j < R::LOADS; ++j) lds_copy_b128_nt(j * R::KEYS < 16 ? half0 : half1, off[j], to + j * 1024);
        } else {
#pragma unroll
            for (int j = 0; j < R::LOADS; ++j) lds_copy_b128(j * R::KEYS < 16 ? half0 : half1, off[j], to + j * 1024);
        }
    };
    auto copy_keys = [&](int stage, const Pages& p) {
        const uint32_t to = ring + stage * R::STAGE;
        const int64_t row0 = max(p.row[0], (int64_t)0), row1 = max(p.row[1], (int64_t)0);
        copy_rows(a.k, koff, to + R::K0, row0, row1);
        if constexpr (E4M3)
            lds_copy_b32((lane < 32 ? a.k_scale : a.v_scale) + (lane & 16 ? row1 : row0) + (lane & 15), to + R::S0);
    };
    auto copy_values = [&](int stage, const Pages& p) {
        copy_rows(a.v, voff, ring + stage * R::STAGE + R::V0, max(p.row[0], (int64_t)0), max(p.row[1], (int64_t)0));
    };

    // this lane's query: 8 elements of every 32
    bf16x8 q[D / 32];
    {
        const int r = min(my_row, item.s.tokens * a.G - 1);
        const int64_t at = ((int64_t)(item.s.first_token + r / a.G) * a.Hq + h * a.G + r % a.G) * D + 8 * g;
#pragma unroll
        for (int ks = 0; ks < D / 32; ++ks) q[ks] = as_bf16x8(*reinterpret_cast<const u32x4*>(a.q + at + 32 * ks));
    }

    Pages held[R::NS];                                   // of the tiles in LDS
#pragma unroll
    for (int s = 0; s < R::NS; ++s)
        if (s < tiles) held[s] = pages_of(key_of(s));
    arrived(q);
#pragma unroll
    for (int s = 0; s < R::NS; ++s)
        if (s < tiles) {
            copy_keys(s, held[s]);
            copy_values(s, held[s]);
        }

    Running run;
    f32x4 o[D / 16];
#pragma unroll
    for (int d = 0; d < D / 16; ++d) o[d] = f32x4{0.f, 0.f, 0.f, 0.f};

    auto step = [&](auto stage, int i) {
        constexpr int S = decltype(stage)::value;
        const Pages here = held[S];
        const bool more = i + R::NS < tiles;
        if (more) held[S] = pages_of(key_of(i + R::NS));
        // behind this tile's keys: its values, and the tiles after it
        wait_behind<R::NS, R::KCOPIES + R::VCOPIES, R::VCOPIES>(tiles - 1 - i);
        const int key0 = key_of(i);
        const uint32_t kb0 = ring + S * R::STAGE + R::K0, vb0 = ring + S * R::STAGE + R::V0, sb0 = ring + S * R::STAGE + R::S0;

        // S^T: lane (c, g) receives keys 16 x + 4 g + r of column c
        float s[8];
        f32x4 vs[2];
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            f32x4 acc = f32x4{0.f, 0.f, 0.f, 0.f};
            const int key = 16 * x + c;
#pragma unroll
            for (int ks = 0; ks < D / 32; ++ks) {
                u32x4 k;
                if constexpr (E4M3)
                    k = e4m3_to_bf16(lds_read<u32x2>(kb0 + key * R::RB + ((2 * ks + (g >> 1)) ^ R::swap_k(key)) * 16 + (g & 1) * 8));
                else
                    k = lds_read<u32x4>(kb0 + key * R::RB + ((4 * ks + g) ^ R::swap_k(key)) * 16);
                acc = mfma_bf16_16x16x32(as_bf16x8(k), q[ks], acc);
            }
            f32x4 factor = f32x4{a.scale2, a.scale2, a.scale2, a.scale2};
            if constexpr (E4M3) {
                factor *= lds_read<f32x4>(sb0 + (16 * x + 4 * g) * 4);
                vs[x] = lds_read<f32x4>(sb0 + 128 + (16 * x + 4 * g) * 4);
            }
#pragma unroll
            for (int r = 0; r < 4; ++r) s[4 * x + r] = acc[r] * factor[r];
        }
        if (more) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the keys have been read
            copy_keys(S, held[S]);
        }

        // which of this lane's keys its row sees
        const bool whole = here.row[0] >= 0 && here.row[1] >= 0 && key0 >= a.prefix && key0 + 31 <= pos_min &&
                           (a.window <= 0 || key0 > pos_max - a.window || key0 + 31 < a.sinks);
        uint32_t seen = 0xff;
        if (!whole) {
            uint64_t m = ~0ull;
            if (a.window > 0) m = ~bits_to(pos - a.window - key0) | bits_to(a.sinks - 1 - key0);
            m &= bits_to(min(pos, limit - 1) - key0) & ~bits_to(a.prefix - 1 - key0);
            if (here.row[0] < 0) m &= ~0xffffull;
            if (here.row[1] < 0) m &= 0xffffull;
            const uint32_t w = (uint32_t)m >> (4 * g);
            seen = (w & 15u) | (w >> 12 & 0xf0u);
#pragma unroll
            for (int e = 0; e < 8; ++e) s[e] = seen >> e & 1 ? s[e] : -__builtin_inff();
        }

        // the running maximum; its lanes are c, c + 16, c + 32, c + 48
        float top = s[0];
#pragma unroll
        for (int e = 1; e < 8; ++e) top = larger(top, s[e]);
        float t2;
        top = both16(top, t2);
        top = larger(top, t2);
        top = both32(top, t2);
        top = larger(top, t2);
        if (__ballot(run.outgrown(top))) {
            const float w = run.follow(top);
#pragma unroll
            for (int d = 0; d < D / 16; ++d) o[d] *= w;
        }
        const float ref = run.reference();
        float p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            p[e] = __builtin_amdgcn_exp2f(s[e] - ref);
            run.l += p[e];
            if constexpr (E4M3) p[e] *= vs[e >> 2][e & 3];
        }
        if constexpr (E4M3)
            if (!whole) {
#pragma unroll
                for (int e = 0; e < 8; ++e) p[e] = seen >> e & 1 ? p[e] : 0.0f;   // whatever its scale
            }
        const u32x4 hi = pack8(p);
        float rest[8];
        unpack8(hi, rest);
        // an infinite product (its scale overflowed) has no rest: the finite number here adds to the infinity
#pragma unroll
        for (int e = 0; e < 8; ++e) rest[e] = E4M3 ? fminf(p[e] - rest[e], 0x1p100f) : p[e] - rest[e];
        const u32x4 lo = pack8(rest);
        wait_behind<R::NS, R::KCOPIES + R::VCOPIES, R::KCOPIES>(tiles - 1 - i, more);

        // V^T: lane (c, g) takes element 16 d + c of keys 4 g .. and 16 + 4 g ..
        auto values = [&](int d) {
            if constexpr (E4M3) {
                const int key = (c >> 3 << 4) + 4 * g + (c >> 1 & 3);
                return e4m3_to_bf16(lds_columns_b8(vb0 + key * R::RB + (d ^ R::swap_v(key)) * 16 + (c & 1) * 8));
            } else {
                const int key = 4 * g + (c >> 2);
                const uint32_t at = vb0 + key * R::RB + ((2 * d + (c >> 1 & 1)) ^ R::swap_v(key)) * 16 + (c & 1) * 8;
                const u32x2 v0 = lds_columns_b16(at), v1 = lds_columns_b16(at + 16 * R::RB);
                return u32x4{v0.x, v0.y, v1.x, v1.y};
            }
        };
        if (whole) {
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                const bf16x8 v = as_bf16x8(values(d));
                o[d] = mfma_bf16_16x16x32(v, as_bf16x8(lo), o[d]);
                o[d] = mfma_bf16_16x16x32(v, as_bf16x8(hi), o[d]);
            }
        } else {
            // by slot: the columns that see it, 16 bits of this lane's group
            uint32_t by[8];
            u32x4 any = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                by[e] = (uint32_t)(__ballot(seen >> e & 1) >> (16 * g)) & 0xffffu;
                any[e >> 1] |= by[e] ? 0xffffu << (16 * (e & 1)) : 0u;
            }
            bool bad = false;
            u32x4 v[D / 16];
#pragma unroll
            for (int d = 0; d < D / 16; ++d) {
                v[d] = values(d) & any;
                bad |= nonfinite8(v[d]);
            }
            if (!__ballot(bad)) {
#pragma unroll
                for (int d = 0; d < D / 16; ++d) {
                    o[d] = mfma_bf16_16x16x32(as_bf16x8(v[d]), as_bf16x8(lo), o[d]);
                    o[d] = mfma_bf16_16x16x32(as_bf16x8(v[d]), as_bf16x8(hi), o[d]);
                }
            } else {
                // column by column, with zeros for what that column does not see
                for (int col = 0; col < 16; ++col) {
                    u32x4 sees = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
                    for (int e = 0; e < 8; ++e) sees[e >> 1] |= by[e] >> col & 1 ? 0xffffu << (16 * (e & 1)) : 0u;
#pragma unroll
                    for (int d = 0; d < D / 16; ++d) {
                        f32x4 r = mfma_bf16_16x16x32(as_bf16x8(v[d] & sees), as_bf16x8(lo), o[d]);
                        r = mfma_bf16_16x16x32(as_bf16x8(v[d] & sees), as_bf16x8(hi), r);
                        if (c == col) o[d] = r;
                    }
                }
            }
        }
        if (more) {
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the values have been read
            copy_values(S, held[S]);
        }
    };
    for (int i = 0; i < tiles; i += R::NS)
        static_for<R::NS>([&](auto s) {
            if (i + decltype(s)::value < tiles) step(s, i + decltype(s)::value);
        });

    // the waves' results meet in LDS, each in its own buffers
    {
        float t2;
        float l = both16(run.l, t2);
        l += t2;
        l = both32(l, t2);
        l += t2;
        float* mine_o = reinterpret_cast<float*>(smem + wave * R::WAVE_BYTES);
#pragma unroll
        for (int d = 0; d < D / 16; ++d) *reinterpret_cast<f32x4*>(mine_o + c * R::OROW + 16 * d + 4 * g) = o[d];
        if (g == 0) {
            mine_o[R::BM * R::OROW + 2 * c] = run.m;
            mine_o[R::BM * R::OROW + 2 * c + 1] = l;
        }
    }
    __syncthreads();
    constexpr int N = D / 16;                            // elements of a thread
    const int r = tid >> 4, d0 = (tid & 15) * N;
    const bool live = r < rows;
    Joined<N> j;
    if (live)
        for (int w = 0; w < R::WAVES; ++w) {
            const float* from = reinterpret_cast<const float*>(smem + w * R::WAVE_BYTES);
            j.add(from[R::BM * R::OROW + 2 * r], from[R::BM * R::OROW + 2 * r + 1], from + r * R::OROW + d0);
        }
    const int own = item.chunks > 1 ? item.chunks : 0;
    const float* slot = a.slots + ((int64_t)item.first * a.Hkv + (int64_t)h * item.chunks) * R::SLOT;
    if (own) {
        if (live) {
            float* to = const_cast<float*>(slot) + (int64_t)item.chunk * R::SLOT;
            store_agent<N>(to + r * D + d0, j.o);
            if (d0 == 0) {
                const float ml[2] = {j.m, j.l};
                store_agent<2>(to + R::BM * D + 2 * r, ml);
            }
        }
        unsigned* counter = a.counters + (int64_t)item.first * a.Hkv + h;
        if (!arrive_and_check_last(counter, own, reinterpret_cast<int*>(smem + R::WAVES * R::WAVE_BYTES))) return;
        if (tid == 0) __hip_atomic_store(counter, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    }
    if (own + a.prior_chunks)
        join_parts<D>(a, smem, h, rows, (int64_t)item.s.first_token * a.G + item.row0, slot, R::SLOT, R::BM * D, own, j);
    if (!live) return;
    const int at = item.row0 + r;
    store_row<N>(a, D, (int64_t)(item.s.first_token + at / a.G) * a.Hq + h * a.G + at % a.G, d0, j);
}

// ---------------------------------------------------------------------------
// Many rows (prefill, several tokens a sequence, a prefix shared by a batch): a
// workgroup takes a row tile of 128, each of its four waves 32 rows, and goes over tiles of 64
// keys that all waves read from LDS, where they are copied straight from the cache, one to
// three tiles ahead.  e4m3 codes become bf16 (exact) as they are read.
//
// Bound by the matrix instructions and, nearly as much, by the exponentials.  A wave multiplies
// the next tile's scores while it takes this one's exponentials (4096 rows of 8192 keys 465 ->
// 425 us; e4m3 525 -> 485), and finds what the next tile needs, its largest score with it, under
// the second product (425 -> 407), which goes before the other workgroup's work where a row has
// 128 elements (400 -> 391, e4m3 473 -> 461; heads of 64 254 -> 263).  Two workgroups on a CU let
// one's softmax run under another's products; heads of 64, with half the products to as many
// exponentials, take three, in 168 registers: what is cheap to find again is not kept over the
// loop (7 ragged chunks under a window of 512 70 -> 59 us; e4m3 with sinks 88 -> 77).  The vector
// units' cycles and the matrix units' add up to about the whole time: 53 and 56 % with 128
// elements, 63 and 37 with 64, e4m3 68 and 41, 75 and 28.  Now 4096 rows of 8192 keys, in a long run
// (short ones, as the steps above, are a few per cent slower): 380 us (1085 TFLOP/s), e4m3 439
// (939); heads of 64 247 (836), e4m3 302 (683).
//
// Probabilities are rounded to bf16 once for the second product: the output is then off by 0.0023
// of its size where its own rounding makes 0.0017.  The pass over a shared prefix does so for
// every row, also of sequences whose own keys the kernel above takes without that loss: the rest
// as a second product would cost 32 / 128 sequences behind 8192 / 16384 tokens 29.8 -> 31.4 us and
// 130 -> 159, 64 of 4 tokens behind 8192 82 -> 96.
// ---------------------------------------------------------------------------
template <int D, bool E4M3>
struct Tiles {
    static constexpr int WAVES = 4, BM = 32 * WAVES, TK = 64;
    static constexpr int RB = E4M3 ? D : 2 * D, PIECES = RB / 16;        // a cached row
    static constexpr int KEYS = 64 / PIECES;             // keys of one copy
    static constexpr int LOADS = 16 / KEYS;              // a wave copies 16 keys and 16 values
    static constexpr int COPIES = 2 * LOADS + (E4M3 ? 1 : 0);
    // a stage: keys, values, with e4m3 256 bytes of a wave's scales (16 of keys, 16 of values), and by wave whether
    // its keys have a page and whether one of its values is not finite
    static constexpr int K0 = 0, V0 = TK * RB, S0 = 2 * TK * RB, LIVE = S0 + (E4M3 ? 256 * WAVES : 0), BAD = LIVE + 16;
    static constexpr int STAGE = (BAD + 16 + 255) / 256 * 256;
    static constexpr int NB = RB == 256 ? 2 : RB == 128 && D == 64 ? 3 : 4;         // stages: one multiplied, the others on their way
    static constexpr int ENDS = NB * STAGE, LDS = ENDS + 8 * WAVES;      // and the waves' first and last positions
    static constexpr int SLOT = BM * (D + 2);            // floats
    // Where a row's 16-byte piece lies: pieces change places by the key so that the lanes of a read meet different banks.
    __device__ static __forceinline__ int swap_k(int key) {
        return PIECES == 16 ? key & 15 : PIECES == 8 ? (key >> 1) & 7 : (key >> 2) & 3;
    }
    __device__ static __forceinline__ int swap_v(int key) {
        if (E4M3) return PIECES == 8 ? (key >> 1 & 1) * 2 + (key >> 3 & 1) * 4 : (key >> 3 & 1) * 2;
        return PIECES == 16 ? (key & 3) * 4 + (key >> 2 & 1) * 2 : (key >> 1 & 1) * 4 + (key >> 2 & 1) * 2;
    }
    // what copy j's offsets differ by from the first copy's, beside 1024 j
    static constexpr int flip_k(int j) { return 64 * j; }
    static constexpr int flip_v(int j) { return E4M3 ? 64 * j : D == 128 ? j % 2 * 32 : 0; }
};

// PREFIX: the rows are all T tokens' and the keys the shared ones; partial results.
template <int D, bool E4M3, bool PREFIX>
__global__ __launch_bounds__(256, D == 64 ? 3 : 2) void attention_tiles_kernel(Call a) {
    using R = Tiles<D, E4M3>;
    extern __shared__ __attribute__((aligned(256))) unsigned char smem[];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int c = lane & 31, hf = lane >> 5;             // column (row of the wave), half
    const int h = blockIdx.x % a.Hkv;
    Item item;
    int total_rows;
    if constexpr (PREFIX) {
        item.chunks = a.target;
        item.chunk_tiles = a.least;
        item.chunk = blockIdx.x / a.Hkv % item.chunks;
        item.row0 = blockIdx.x / a.Hkv / item.chunks * R::BM;
        item.b = 0;
        item.s = Sequence{0, a.T, a.prefix};
        total_rows = a.T * a.G;
    } else {
        if (!find_item<R::BM, R::TK, true>(a, (int)(blockIdx.x / a.Hkv), item)) return;
        total_rows = item.s.tokens * a.G;
    }
    const int my_row = item.row0 + 32 * wave + c;
    const bool mine = my_row < total_rows;
    const int token = item.s.first_token + min(my_row, total_rows - 1) / a.G;
    const int head = h * a.G + min(my_row, total_rows - 1) % a.G;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) unsigned char*)smem;
    // this row's position (-1 sees nothing), and the first and last of the wave's and of the workgroup's rows that exist
    int pos = -1, pos_min, pos_max, all_min, all_max;
    if constexpr (PREFIX) {
        // the last offset that is not above the token
        int lo = 0, hi = a.B;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (a.q_offsets[mid] <= token) lo = mid;
            else hi = mid - 1;
        }
        if (mine && lo < a.B) {
            const Sequence s = sequence_of(a.q_offsets[lo], a.q_offsets[lo + 1], a.kv_len[lo], a.T);
            if (token >= s.first_token && token < s.first_token + s.tokens) pos = max(s.len - s.tokens + token - s.first_token, -1);
        }
        pos_min = mine ? pos : 0x7fffffff;
        pos_max = mine ? pos : -1;
#pragma unroll
        for (int o = 1; o < 64; o <<= 1) {
            pos_min = min(pos_min, __shfl_xor(pos_min, o, 64));
            pos_max = max(pos_max, __shfl_xor(pos_max, o, 64));
        }
        all_min = pos_min = __builtin_amdgcn_readfirstlane(pos_min);
        all_max = pos_max = __builtin_amdgcn_readfirstlane(pos_max);
        if (lane == 0) lds_write(lds0 + R::ENDS + 8 * wave, i32x2{pos_min, pos_max});
        __syncthreads();
        for (int w = 0; w < R::WAVES; ++w) {
            const i32x2 ends = lds_read<i32x2>(lds0 + R::ENDS + 8 * w);
            all_min = min(all_min, __builtin_amdgcn_readfirstlane(ends[0]));
            all_max = max(all_max, __builtin_amdgcn_readfirstlane(ends[1]));
        }
    } else {
        // rows are in order of position: lanes 0 .. 3 find the ends
        const int before = item.s.len - item.s.tokens, first = item.row0 + 32 * wave;
        if (mine) pos = max(before + token - item.s.first_token, -1);
        const int end = min((lane & 1 ? first : item.row0) + (lane & 1 ? 31 : lane & 2 ? R::BM - 1 : 0), total_rows - 1);
        const int ends = max(before + end / a.G, -1);
        pos_min = first < total_rows ? __builtin_amdgcn_readfirstlane(pos) : 0x7fffffff;
        pos_max = first < total_rows ? __builtin_amdgcn_readlane(ends, 1) : -1;
        all_min = __builtin_amdgcn_readlane(ends, 0);
        all_max = __builtin_amdgcn_readlane(ends, 2);
    }
    const int key_begin = PREFIX ? 0 : a.prefix;
    const int limit = PREFIX ? a.prefix : (int)min((int64_t)item.s.len, (int64_t)a.max_pages << a.page_shift);

    // the tiles: a chunk of the sequence's, less those that lie ahead of the whole row tile
    int i0 = 0, tiles;
    if constexpr (PREFIX) {
        item.span = Span{0, 0, 0, (a.prefix + R::TK - 1) / R::TK};
        i0 = item.chunk * item.chunk_tiles;
        tiles = min(item.chunk_tiles, item.span.n - i0);
    } else {
        if (item.chunks > 1) {
            i0 = item.chunk * item.chunk_tiles;
            tiles = min(item.chunk_tiles, item.span.n - i0);
            while (tiles > 0 && item.span.tile(i0 + tiles - 1) * R::TK > all_max) --tiles;
        } else {
            item.span = span_of<R::TK>(a, Sequence{0, all_max - all_min + 1, max(all_max + 1, 0)});
            tiles = item.span.n;
        }
    }

    // a wave brings 16 keys of every tile; the first copy's offsets from their first row
    uint32_t koff = lane / R::PIECES * R::RB + ((lane % R::PIECES) ^ R::swap_k(lane / R::PIECES)) * 16;
    uint32_t voff = lane / R::PIECES * R::RB + ((lane % R::PIECES) ^ R::swap_v(lane / R::PIECES)) * 16;
    const uint32_t page_bytes = ((uint32_t)a.Hkv << a.page_shift) * R::RB;
    const unsigned char* keys = static_cast<const unsigned char*>(a.k) + ((int64_t)h << a.page_shift) * R::RB;
    const unsigned char* values = static_cast<const unsigned char*>(a.v) + ((int64_t)h << a.page_shift) * R::RB;
    // the first of the wave's keys of a tile, and their page (any entry of the table past the end)
    auto key_of = [&](int i) { return item.span.tile(i0 + i) * R::TK + 16 * wave; };
    auto page_of = [&](int key) {
        const int64_t b = PREFIX || key < a.shared ? 0 : item.b;
        return load_scalar(a.table + b * a.max_pages + min(key >> a.page_shift, a.max_pages - 1));
    };
    // where they lie in the cache (without a page: anywhere in it)
    struct Place {
        int64_t at;
        bool paged;
    };
    auto place_of = [&](int key, int page) {
        const bool paged = key < limit && (unsigned)page < (unsigned)a.pages;
        return Place{(int64_t)(paged ? page : 0) * page_bytes + (key & ((1 << a.page_shift) - 1)) * R::RB, paged};
    };
    bool all_paged = true;                               // whether every key of the item has a page; found below
    auto copy_keys = [&](uint32_t stage, const Place& p) {
#pragma unroll
        for (int j = 0; j < R::LOADS; ++j)
            lds_copy_b128(keys + p.at, (koff ^ R::flip_k(j)) + 1024 * j, stage + R::K0 + 16 * wave * R::RB + j * 1024);
    };
    auto copy_values = [&](uint32_t stage, const Place& p) {
#pragma unroll
        for (int j = 0; j < R::LOADS; ++j)
            lds_copy_b128(values + p.at, (voff ^ R::flip_v(j)) + 1024 * j, stage + R::V0 + 16 * wave * R::RB + j * 1024);
        if constexpr (E4M3) {
            const int64_t row = ((int64_t)h << a.page_shift) + p.at / R::RB;
            lds_copy_b32((lane & 16 ? a.v_scale : a.k_scale) + row + (lane & 15), stage + R::S0 + 256 * wave);
        }
        if (!all_paged && lane == 0) lds_write<int>(stage + R::LIVE + 4 * wave, p.paged);
    };
    // the tiles that rows from position `first` to `last` see all of
    struct Whole {
        int lo, n, sink_lo, sink_n;
        __device__ __forceinline__ bool has(int tile) const {
            return (unsigned)(tile - lo) < (unsigned)n || (unsigned)(tile - sink_lo) < (unsigned)sink_n;
        }
    };
    auto whole_for = [&](int first, int last) {
        const int begin = (key_begin + R::TK - 1) / R::TK, end = (min(limit - 1, first) + 1) / R::TK;
        Whole w;
        w.lo = a.window > 0 && last >= a.window ? max((last - a.window) / R::TK + 1, begin) : begin;
        w.n = max(end - w.lo, 0);
        w.sink_lo = begin;
        w.sink_n = a.window > 0 ? max(min(end, a.sinks / R::TK) - begin, 0) : 0;
        return w;
    };
    const Whole all_whole = whole_for(all_min, all_max);

    // a lane's place in a tile: its key's row with the first of its pieces, from which that of another step of
    // keys and block of values is an exclusive or away (stages and rows are multiples of what it changes)
    uint32_t kat = R::K0 + c * R::RB + (E4M3 ? R::swap_k(c) * 16 + hf * 8 : (hf ^ R::swap_k(c)) * 16);
    const int vkey = E4M3 ? 4 * hf + (lane >> 1 & 3) + (lane >> 3 & 1) * 8 : 4 * hf + (lane >> 2 & 3);
    const int vpiece = E4M3 ? c >> 4 : 2 * (c >> 4) + (lane >> 1 & 1);
    uint32_t vat = R::V0 + vkey * R::RB + (vpiece ^ R::swap_v(vkey)) * 16 + (lane & 1) * 8;
    uint32_t sat = R::S0 + 16 * hf;                      // scales of keys 8 j + 4 hf ..: 256 (j / 2) + 32 (j % 2) on, of values 64 behind

    // This lane's query: 8 elements of every 16, times the sign of the scale, or zero for a scale of zero (exact; masked
    // scores are minus infinity before they are scaled, and zero times that would be NaN).
    bf16x8 q[D / 16];
    {
        const uint16_t* from = a.q + ((int64_t)token * a.Hq + head) * D + 8 * hf;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) q[ks] = as_bf16x8(*reinterpret_cast<const u32x4*>(from + 16 * ks));
        if (a.scale2 <= 0.0f) {
            const float sign = a.scale2 < 0.0f ? -1.0f : 0.0f;
#pragma unroll
            for (int ks = 0; ks < D / 16; ++ks) {
                float f[8];
                unpack8(__builtin_bit_cast(u32x4, q[ks]), f);
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] *= sign;
                q[ks] = as_bf16x8(pack8(f));
            }
        }
    }
    const float scale2 = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(a.scale2 == 0.0f ? 1.0f : fabsf(a.scale2))));

    // A stage holds a tile's values and the next tile's keys: while the softmax of a tile runs,
    // the next one's scores are multiplied.
    constexpr int FAR = R::NB - 1;                       // stages on their way
    int page[FAR + 3];
#pragma unroll
    for (int i = 0; i < FAR + 3; ++i) page[i] = page_of(key_of(i));
    for (int j = lane; j < 4 * tiles; j += 64) {         // 16 keys of the item, by lane, while the query is on its way
        const int key = item.span.tile(i0 + (j >> 2)) * R::TK + 16 * (j & 3);
        const int64_t b = PREFIX || key < a.shared ? 0 : item.b;
        const int id = a.table[b * a.max_pages + min(key >> a.page_shift, a.max_pages - 1)];
        if (key < limit && (unsigned)id >= (unsigned)a.pages) all_paged = false;
    }
    all_paged = __ballot(!all_paged) == 0;
    arrived(q);
    uint32_t stage = lds0, behind = lds0 + FAR * R::STAGE;
    Place place = place_of(key_of(0), page[0]);          // of the tile whose values are copied next, and of the one after it
    if (tiles > 0) copy_keys(behind, place);
    Place after = place_of(key_of(1), page[1]);
#pragma unroll
    for (int i = 0; i < FAR; ++i) {
        if (i < tiles) {
            copy_keys(lds0 + i * R::STAGE, after);
            copy_values(lds0 + i * R::STAGE, place);
        }
        place = after;
        after = place_of(key_of(i + 2), page[i + 2]);
    }
    int next_key = key_of(FAR + 2), next = page[FAR + 2];
    int tile = item.span.tile(i0);
    bool plain = all_paged && all_whole.has(tile);       // every row sees all of the tile
    // what the next tile needs, found under this one's products
    auto ahead = [&](int i) {
        place = after;
        after = place_of(next_key, next);
        tile = item.span.tile(i0 + i + 1);
        plain = all_paged && all_whole.has(tile);
    };

    Running run;
    f32x16 o[D / 32];
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) o[d][e] = 0.0f;
    f32x16 odd_o[D / 32];                                // the sums of tiles whose values are not all finite, if
    in_memory(odd_o);
    bool any_odd = false;                                // there is one

    // S^T of the keys in a stage: lane (c, hf) receives keys 32 x + 8 (e / 4) + 4 hf + e % 4 of column c.
    // Product n takes elements n / 2 of keys 32 (n % 2) ..; its keys are on their way AHEAD products before.
    constexpr int N = D / 8, AHEAD = D == 64 ? 3 : 4;    // (3: registers)
    using Fragment = std::conditional_t<E4M3, u32x2, u32x4>;
    auto bf16_of = [&](Fragment f) {
        if constexpr (E4M3) return as_bf16x8(e4m3_to_bf16(f));
        else return as_bf16x8(f);
    };
    auto key_fragment = [&](uint32_t stage, int n) {
        return lds_read<Fragment>(((stage + kat) ^ (n / 2 * (E4M3 ? 16 : 32))) + n % 2 * 32 * R::RB);
    };
    // V^T: lane (c, hf) takes element 32 d + c of keys 16 y + 4 hf .. and 16 y + 8 + 4 hf ..
    auto value_fragment = [&](uint32_t stage, int d, int y) -> Fragment {
        if constexpr (E4M3) {
            return lds_columns_b8(((stage + vat) ^ (32 * d)) + 16 * y * R::RB);
        } else {
            const uint32_t at = ((stage + vat) ^ (64 * d)) + 16 * y * R::RB;
            const u32x2 v0 = lds_columns_b16(at), v1 = lds_columns_b16(at + 8 * R::RB);
            return u32x4{v0.x, v0.y, v1.x, v1.y};
        }
    };
    auto scores = [&](uint32_t stage, f32x16 (&s)[2]) {
        Fragment k[AHEAD];
        static_for<AHEAD>([&](auto n) { k[n] = key_fragment(stage, n); });
        static_for<2>([&](auto x) { s[x] = f32x16{}; });
        __builtin_amdgcn_sched_barrier(0);
        static_for<N>([&](auto n_) {
            constexpr int n = decltype(n_)::value;
            s[n % 2] = mfma_bf16_32x32x16(bf16_of(k[n % AHEAD]), q[n / 2], s[n % 2]);
            if constexpr (n + AHEAD < N) k[n % AHEAD] = key_fragment(stage, n + AHEAD);
            __builtin_amdgcn_sched_barrier(0);
        });
    };
    // The lane's largest score, in eight steps.
    float peak;
    auto peaks = [&](int j, const f32x16 (&s)[2]) {
        const float a = larger(s[j / 4][4 * (j % 4)], s[j / 4][4 * (j % 4) + 1]), b = larger(s[j / 4][4 * (j % 4) + 2], s[j / 4][4 * (j % 4) + 3]);
        peak = j == 0 ? larger(a, b) : larger(peak, larger(a, b));
    };
    auto all_peaks = [&](const f32x16 (&s)[2]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) peaks(j, s);
    };
    // one tile: its scores s, the next tile's s2
    auto step = [&](int i, f32x16 (&s)[2], f32x16 (&s2)[2]) {
        // (what follows from these is computed anew in every tile: kept, it takes registers from the products)
        asm volatile("" : "+v"(kat), "+v"(vat), "+v"(sat), "+v"(koff), "+v"(voff));
        wait_tiles<R::COPIES, R::NB - 2>(tiles - 1 - i);
        __syncthreads();                                 // this stage has arrived, and every wave is done with the one behind
        if (i + FAR < tiles) {
            copy_keys(behind, after);
            copy_values(behind, place);
        }
        const int key0 = tile * R::TK;
        i32x4 live4{1, 1, 1, 1};
        bool whole = plain, useful = pos_max >= 0;
        if (!plain) {
            if (!all_paged) live4 = lds_read<i32x4>(stage + R::LIVE);
            whole = __builtin_amdgcn_readfirstlane(live4[0] & live4[1] & live4[2] & live4[3]) && whole_for(pos_min, pos_max).has(tile);
            useful = key0 <= pos_max && (a.window <= 0 || key0 + R::TK > pos_min - a.window || key0 < a.sinks);
            // Where a row of the workgroup does not see all keys: values of positions that hold no key become zeros
            // (a wave its own 16), and a NaN or infinity among the others is found.
            const bool paged = live4[wave] != 0;
            bool odd = false;
            int lane = tid & 63;
            asm volatile("" : "+v"(lane));               // (see above)
            u32x4 zeros{};
            asm volatile("" : "+v"(zeros));
#pragma unroll
            for (int j = 0; j < R::LOADS; ++j) {
                const int key = 16 * wave + j * R::KEYS + lane / R::PIECES;
                const uint32_t at = stage + R::V0 + 16 * wave * R::RB + j * 1024 + 16 * lane;
                if (paged && key0 + key < limit) {
                    const u32x4 v = lds_read<u32x4>(at);
                    if constexpr (E4M3) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) odd |= (((v[e] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) != 0;
                    } else {
                        odd |= nonfinite8(v);
                    }
                } else {
                    lds_write(at, zeros);
                }
            }
            if (E4M3 && lane < 16) {
                const uint32_t at = stage + R::S0 + 256 * wave + 64 + 4 * lane;
                if (paged && key0 + 16 * wave + lane < limit) odd |= !__builtin_isfinite(lds_read<float>(at));
                else lds_write(at, 0.0f);
            }
            const uint64_t some = __ballot(odd);
            if (lane == 0) lds_write<int>(stage + R::BAD + 4 * wave, some != 0);
            __syncthreads();
        }
        // the keys of the tile that this lane's row sees
        const auto seen_keys = [&] {
            uint64_t m = ~0ull;
            if (a.window > 0) m = ~bits_to(pos - a.window - key0) | bits_to(a.sinks - 1 - key0);
            m &= bits_to(min(pos, limit - 1) - key0) & ~bits_to(key_begin - 1 - key0);
#pragma unroll
            for (int w = 0; w < R::WAVES; ++w)
                if (!__builtin_amdgcn_readfirstlane(live4[w])) m &= ~(0xffffull << (16 * w));
            return m;
        };
        if (useful) {
            if constexpr (E4M3) {
                f32x4 k[8];
                static_for<8>([&](auto j) { k[j] = lds_read<f32x4>(stage + sat + j / 2 * 256 + j % 2 * 32); });
#pragma unroll
                for (int j = 0; j < 8; ++j)
#pragma unroll
                    for (int r = 0; r < 4; ++r) s[j / 4][4 * (j % 4) + r] *= k[j][r];
            }
            if (!whole) {
                const uint64_t seen = seen_keys() >> (4 * hf);       // its half's first key in bit 0
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const uint32_t w = (uint32_t)(seen >> (32 * x));
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        int sees = __builtin_amdgcn_sbfe((int)w, 8 * (e >> 2) + (e & 3), 1);     // 0 or -1
                        asm("" : "+v"(sees));
                        s[x][e] = __int_as_float((__float_as_int(s[x][e]) & sees) | (0xff800000 & ~sees));
                    }
                }
            }
            if (E4M3 || !whole) all_peaks(s);
            float t2;
            float top = both32(peak, t2);
            top = larger(top, t2) * scale2;
            if (__ballot(run.outgrown(top))) {
                const float w = run.follow(top);
#pragma unroll
                for (int d = 0; d < D / 32; ++d) o[d] *= w;
                if (any_odd)
#pragma unroll 1
                    for (int d = 0; d < D / 32; ++d) odd_o[d] *= w;
            }
            const float ref = run.reference();
            // P^T: the operand of 16 keys is eight neighbouring results
            u32x4 p[4];
            Fragment ring[AHEAD];                        // keys, then values
            float f[8];
            f32x4 scale;                                 // of values, with e4m3: the next four keys'
            if constexpr (E4M3) scale = lds_read<f32x4>(stage + sat + 64);
            static_for<AHEAD>([&](auto n) { ring[n] = key_fragment(stage, n); });
            static_for<2>([&](auto x) { s2[x] = f32x16{}; });
            __builtin_amdgcn_sched_barrier(0);
            static_for<N>([&](auto n_) {
                constexpr int n = decltype(n_)::value, EACH = 32 / N;
                s2[n % 2] = mfma_bf16_32x32x16(bf16_of(ring[n % AHEAD]), q[n / 2], s2[n % 2]);
                if constexpr (n + AHEAD < N) ring[n % AHEAD] = key_fragment(stage, n + AHEAD);
                static_for<EACH>([&](auto j) {
                    constexpr int e = n * EACH + decltype(j)::value;
                    f[e % 8] = __builtin_amdgcn_exp2f(fmaf(s[e / 16][e % 16], scale2, -ref));
                    run.l += f[e % 8];
                    if constexpr (E4M3 && e % 4 == 3) {
                        constexpr int next = e / 4 + 1;
#pragma unroll
                        for (int r = 0; r < 4; ++r) f[e % 8 - 3 + r] *= scale[r];
                        if constexpr (next < 8) scale = lds_read<f32x4>(stage + sat + 64 + next / 2 * 256 + next % 2 * 32);
                    }
                    if constexpr (e % 8 == 7) p[e / 8] = pack8(f);
                });
                asm volatile("" : "+v"(run.l));          // (added here, or the terms stay in registers)
                __builtin_amdgcn_sched_barrier(0);
            });
            bool bad = false;
            if (!whole) {
                const i32x4 found = lds_read<i32x4>(stage + R::BAD);
                bad = __builtin_amdgcn_readfirstlane(found[0] | found[1] | found[2] | found[3]) != 0;
            }
            if (!bad) {
                if constexpr (D == 128) __builtin_amdgcn_s_setprio(1);   // (see Tiles)
                static_for<AHEAD>([&](auto n) { ring[n] = value_fragment(stage, n % (D / 32), n / (D / 32)); });
                __builtin_amdgcn_sched_barrier(0);
                static_for<N>([&](auto n_) {
                    constexpr int n = decltype(n_)::value, BLOCKS = D / 32;
                    o[n % BLOCKS] = mfma_bf16_32x32x16(bf16_of(ring[n % AHEAD]), as_bf16x8(p[n / BLOCKS]), o[n % BLOCKS]);
                    if constexpr (n + AHEAD < N) ring[n % AHEAD] = value_fragment(stage, (n + AHEAD) % BLOCKS, (n + AHEAD) / BLOCKS);
                    if constexpr (n == AHEAD) ahead(i);
                    if constexpr (!E4M3 && n % (N / 8) == 0) peaks(n / (N / 8), s2);
                    __builtin_amdgcn_sched_barrier(0);
                });
                if constexpr (D == 128) __builtin_amdgcn_s_setprio(0);
            } else {
                // Key by key, and nothing of a key that the column does not see.  These sums and the probabilities are
                // kept in memory: the registers are the other path's.
                u32x4 parked[4];
                in_memory(parked);
#pragma unroll
                for (int y = 0; y < 4; ++y) parked[y] = p[y];
                in_memory(parked);
                const uint64_t seen = seen_keys();
#pragma unroll 1
                for (int d = 0; d < D / 32; ++d) {
                    f32x16 sum{};
                    if (any_odd) sum = odd_o[d];
#pragma unroll 1
                    for (int key = 0; key < R::TK; ++key) {
                        // in the half (key / 4) % 2 of its operand
                        const uint32_t two = parked[key >> 4][(key >> 3 & 1) * 2 + (key >> 1 & 1)];
                        float upper;
                        const float lower = both32(__uint_as_float(key & 1 ? two & 0xffff0000u : two << 16), upper);
                        const float prob = key & 4 ? upper : lower;
                        const bool sees = seen >> key & 1;
                        const uint32_t row = stage + R::V0 + key * R::RB;
#pragma unroll
                        for (int y = 0; y < 4; ++y) {
                            u32x2 v;                     // elements 32 d + 8 y + 4 hf ..
                            if constexpr (E4M3) {
                                const u32x4 w = e4m3_to_bf16(
                                    u32x2{lds_read<uint32_t>(row + ((2 * d + y / 2) ^ R::swap_v(key)) * 16 + y % 2 * 8 + 4 * hf), 0u});
                                v = u32x2{w.x, w.y};
                            } else {
                                v = lds_read<u32x2>(row + ((4 * d + y) ^ R::swap_v(key)) * 16 + 8 * hf);
                            }
#pragma unroll
                            for (int r = 0; r < 4; ++r) {
                                const float with = fmaf(prob, __uint_as_float(r & 1 ? v[r / 2] & 0xffff0000u : v[r / 2] << 16), sum[4 * y + r]);
                                sum[4 * y + r] = sees ? with : sum[4 * y + r];
                            }
                        }
                    }
                    odd_o[d] = sum;
                }
                in_memory(odd_o);
                any_odd = true;
                all_peaks(s2);
                ahead(i);
            }
        } else {
            if (i + 1 < tiles) {
                scores(stage, s2);
                all_peaks(s2);
            }
            ahead(i);
        }
        next_key = key_of(i + FAR + 3);
        next = page_of(next_key);                        // on its way while the waves gather (LDS reads would wait for it)
        behind = stage;
        stage = stage == lds0 + FAR * R::STAGE ? lds0 : stage + R::STAGE;
    };
    if (tiles > 0) {
        f32x16 even[2], odd[2];
        wait_tiles<R::COPIES, FAR>(tiles);
        __syncthreads();
        scores(behind, even);
        all_peaks(even);
        for (int i = 0;;) {
            step(i, even, odd);
            if (++i == tiles) break;
            step(i, odd, even);
            if (++i == tiles) break;
        }
    }

    if (any_odd)
#pragma unroll
        for (int d = 0; d < D / 32; ++d) o[d] += odd_o[d];
    float t2;
    float l = both32(run.l, t2);
    l += t2;
    const float m = run.m;
    // element 32 d + 8 y + 4 hf + r of the row is o[d][4 y + r]
    if constexpr (PREFIX) {
        if (!mine) return;
        const int64_t row = ((int64_t)item.chunk * a.Hkv + h) * total_rows + my_row;
        float* to = a.prior + row * D + 4 * hf;
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
#pragma unroll
            for (int y = 0; y < 4; ++y)
                *reinterpret_cast<f32x4*>(to + 32 * d + 8 * y) = f32x4{o[d][4 * y], o[d][4 * y + 1], o[d][4 * y + 2], o[d][4 * y + 3]};
        if (hf == 0) *reinterpret_cast<f32x2*>(a.prior_ml + 2 * row) = f32x2{m, l};
        return;
    }
    if (!mine) return;
    int again = threadIdx.x;                             // the row once more: kept over the loop it would take registers
    asm volatile("" : "+v"(again));
    if (item.chunks > 1 || a.prior_chunks) {             // a part: attention_join_kernel joins them
        const int r = 32 * wave + (again & 31);
        float* slot = a.slots + ((int64_t)item.first * a.Hkv + (int64_t)h * item.chunks + item.chunk) * R::SLOT;
#pragma unroll
        for (int d = 0; d < D / 32; ++d)
#pragma unroll
            for (int y = 0; y < 4; ++y)
                *reinterpret_cast<f32x4*>(slot + r * D + 32 * d + 8 * y + 4 * hf) =
                    f32x4{o[d][4 * y], o[d][4 * y + 1], o[d][4 * y + 2], o[d][4 * y + 3]};
        if (hf == 0) *reinterpret_cast<f32x2*>(slot + R::BM * D + 2 * r) = f32x2{m, l};
        return;
    }
    const int its = item.row0 + 32 * wave + (again & 31);
    const int64_t row = (int64_t)(item.s.first_token + its / a.G) * a.Hq + h * a.G + its % a.G;
    // the halves exchange, so that a lane stores eight neighbouring elements
#pragma unroll
    for (int d = 0; d < D / 32; ++d)
#pragma unroll
        for (int y = 0; y < 4; y += 2) {
            uint32_t w[2][2];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                Joined<4> j;
                j.l = l;
#pragma unroll
                for (int r = 0; r < 4; ++r) j.o[r] = o[d][4 * (y + x) + r];
                rounded<4>(j, w[x]);
            }
            const auto first = __builtin_amdgcn_permlane32_swap(w[0][0], w[1][0], false, false);
            const auto second = __builtin_amdgcn_permlane32_swap(w[0][1], w[1][1], false, false);
            *reinterpret_cast<u32x4*>(a.out + row * D + 32 * d + 8 * (y + hf)) = u32x4{first[0], second[0], first[1], second[1]};
        }
    if (a.lse && hf == 0) a.lse[row] = lse_of(m, l);
}

// Joins the parts that attention_tiles_kernel left: 16 rows of a row tile a workgroup, so
// that the parts' 66 KB of each tile and chunk are read by many CUs (joined by the last
// workgroup of a tile, 64 chunks took 120 us).  Row tiles are the grid's y and z: along x
// alone a large batch behind a shared prefix would have 2^32 threads and more.
template <int D>
__global__ __launch_bounds__(256) void attention_join_kernel(Call a) {
    using R = Tiles<D, false>;
    __shared__ __attribute__((aligned(16))) unsigned char smem[kJoinBytes<D>];
    const int h = blockIdx.x % a.Hkv, group = blockIdx.x / a.Hkv;
    Item item;
    if (!find_item<R::BM, R::TK, true, true>(a, (int)(blockIdx.y + gridDim.y * blockIdx.z), item)) return;
    if (item.chunks == 1 && !a.prior_chunks) return;     // written already
    const int row0 = item.row0 + 16 * group;
    const int rows = min(16, item.s.tokens * a.G - row0);
    if (rows <= 0) return;
    const float* slot = a.slots + ((int64_t)item.first * a.Hkv + (int64_t)h * item.chunks) * R::SLOT + 16 * group * D;
    constexpr int N = D / 16;
    Joined<N> j;
    join_parts<D>(a, smem, h, rows, (int64_t)item.s.first_token * a.G + row0, slot, R::SLOT,
                  R::BM * D - 16 * group * D + 2 * 16 * group, item.chunks, j);
    const int r = threadIdx.x >> 4, at = row0 + r;
    if (r < rows)
        store_row<N>(a, D, (int64_t)(item.s.first_token + at / a.G) * a.Hq + h * a.G + at % a.G, (threadIdx.x & 15) * N, j);
}

// ---------------------------------------------------------------------------
// The plan of a call, from its sizes alone.
// ---------------------------------------------------------------------------
struct Plan {
    bool rows, tiles, join;      // which kernels run
    int few_rows;                // of a sequence, for the first of them
    int row_items, row_target, row_least;        // their work items for each key head at most; chunks wanted (0: keys are
    int tile_items, tile_target, tile_tiles;     // not split) and key tiles of one at least; row tiles
    int prior_chunks, prior_tiles;               // of the shared prefix: chunks, and key tiles of one
    bool stream;
    size_t slots, prior;         // floats
    size_t bytes() const { return slots + prior ? kCounterBytes + (slots + prior) * 4 : 0; }
};

Plan plan_of(int T, int B, int64_t max_kv, int Hq, int Hkv, int D, bool e4m3, int prefix, int max_q) {
    const int64_t G = Hq / Hkv, all = (int64_t)T * G;
    const int64_t cus = device_cu_count();
    const int64_t most_rows = max_q > 0 ? std::min(all, max_q * G) : all;        // of a sequence
    Plan p{};
    // A shared prefix is worth a pass of its own from 64 MB of rereading on (that pass and its partial results cost about
    // 12 us), and while a sequence has fewer rows than a row tile: the rows of a prompt fill tiles by themselves, to which a
    // pass adds only partial results.  16 sequences of 4 / 64 / 128 / 256 / 1024 rows behind 8192 tokens with a pass 22 / 56 /
    // 92 / 161 / 590 us, without 46 / 72 / 86 / 148 / 511; 32 behind 2048 with 21 / 46 / 76 / 115 / 462, without 31 / 47 / 51 /
    // 76 / 302.
    if ((int64_t)(B - 1) * prefix * Hkv * D * 4 < (int64_t)64 << 20 || all >= 128 * (int64_t)B) prefix = 0;
    const int64_t own = max_kv - prefix;
    // Sequences of few rows stream their keys once for every 16 rows, more are worth tiles of 128: few is 16 rows, and up to
    // 128 where that is little work, 3/4 of a million keys, heads and row tiles in all.  On rows and on tiles: one sequence
    // of 8192 keys with 32 / 64 / 128 rows 19.5 / 21 / 29 us and 28.5 / 30 / 33; 64 of up to 600 with 32 rows 21 and 31, with
    // 48 rows 33 and 38; 8 of 4096 with 64 rows 48 and 40 (e4m3); 64 of 8192 with 32 rows 505 and 365.  A ragged batch
    // (fewer tokens than B times the largest count) holds both.
    p.few_rows = 16 * (int)std::clamp<int64_t>((3 << 18) / std::max<int64_t>(1, (int64_t)B * own * Hkv), 1, 8);
    p.rows = most_rows <= p.few_rows;
    p.tiles = !p.rows;
    if (p.tiles && B > 1 && !(max_q > 0 && (int64_t)max_q * B == T)) p.rows = true;
    if (p.rows) {
        int64_t tiles = std::min(all, all / 16 + B);
        if (p.tiles) tiles = std::min<int64_t>(tiles, (int64_t)B * (p.few_rows / 16));
        // Keys are split while the row tiles do not fill the GPU: into chunks of at least 256 keys for one workgroup a CU;
        // from a row tile a CU on into finer ones of at least 1024 keys, which even out lengths.
        const bool few = tiles * Hkv < cus;
        const int64_t want = std::clamp<int64_t>((few ? 1 : 4) * cus / Hkv, 1, 160);
        p.row_items = (int)tiles;
        p.row_least = few ? 2 : 8;
        if (tiles < want && own > 128 * p.row_least && (tiles + want) * Hkv <= kMaxCounters) {
            p.row_target = (int)want;
            p.row_items = (int)(tiles + want);
            p.slots = (size_t)p.row_items * Hkv * 16 * (D + 2);
        }
        // Read once, past the caches, where they cannot hold it: 64 x 8192 keys 356 -> 317 us (6.0 -> 6.8 TB/s), e4m3 196 -> 172;
        // 67 MB that the caches did hold 21.0 -> 22.7
        p.stream = most_rows <= 16 && (int64_t)B * own * Hkv * D * (e4m3 ? 2 : 4) > (int64_t)128 << 20;
    }
    if (p.tiles) {
        const int64_t tiles = std::min(all, all / 128 + B);
        const int64_t want = std::clamp<int64_t>(2 * cus / Hkv, 1, 160);
        // Where the other kernel takes the sequences of few rows, only so many are left, and partial results are for these
        // (1000 tokens of as many sequences behind 8192 shared positions, 32 heads over 8 of 128: 582 -> 175 MB).
        const int64_t left = p.rows ? std::min(tiles, all / 128 + all / (p.few_rows + 1)) : tiles;
        p.tile_items = p.tile_tiles = (int)left;
        if (tiles < want && own > 256) {
            p.tile_target = (int)want;
            p.tile_items = (int)(left + want);
        }
        p.join = p.tile_target || prefix > 0;
        if (p.join) p.slots = std::max(p.slots, (size_t)p.tile_items * Hkv * 128 * (D + 2));
    }
    if (prefix > 0) {
        // Chunks for two workgroups a CU, of four tiles at least: their partial results are read once more (32 sequences
        // behind 8192 tokens with 2 / 3 / 4 / 6 / 8 tiles 36.7 / 34.4 / 29.7 / 30.4 / 31.1 us).
        const int64_t tiles = (prefix + 63) / 64, rows = (all + 127) / 128;
        const int64_t chunks = std::clamp<int64_t>(2 * cus / (rows * Hkv), 1, std::min<int64_t>((tiles + 3) / 4, 64));
        p.prior_tiles = (int)((tiles + chunks - 1) / chunks);
        p.prior_chunks = (int)((tiles + p.prior_tiles - 1) / p.prior_tiles);
        p.prior = (size_t)p.prior_chunks * Hkv * all * (D + 2);
    }
    return p;
}

template <class Kernel>
void launch(Kernel* kernel, std::atomic<uint64_t>& done, int64_t workgroups, int lds, const Call& a, hipStream_t st) {
    allow_dynamic_lds(reinterpret_cast<const void*>(kernel), lds, done);
    kernel<<<dim3((unsigned)workgroups), 256, lds, st>>>(a);
}

template <int D, bool E4M3>
void launch_all(Call a, const Plan& p, void* ws, hipStream_t st) {
    using R = Rows<D, E4M3>;
    using M = Tiles<D, E4M3>;
    static std::atomic<uint64_t> rows_done{0}, tiles_done{0}, prior_done{0};
    a.counters = static_cast<unsigned*>(ws);
    a.slots = reinterpret_cast<float*>(static_cast<unsigned char*>(ws) + kCounterBytes);
    a.prior = a.slots + p.slots;
    const int64_t rows = (int64_t)a.T * a.G;
    a.prior_ml = a.prior + (size_t)p.prior_chunks * a.Hkv * rows * D;
    if (p.prior_chunks) {
        Call c = a;
        c.target = p.prior_chunks;
        c.least = p.prior_tiles;
        launch(&attention_tiles_kernel<D, E4M3, true>, prior_done, (rows + M::BM - 1) / M::BM * p.prior_chunks * a.Hkv, M::LDS, c, st);
    }
    a.prior_chunks = p.prior_chunks;
    a.few_rows = p.few_rows;
    if (p.tiles) {
        Call c = a;
        c.few = p.rows ? 0 : -1;
        c.items = p.tile_items;
        c.target = p.tile_target;
        c.least = 4;
        launch(&attention_tiles_kernel<D, E4M3, false>, tiles_done, (int64_t)c.items * a.Hkv, M::LDS, c, st);
        if (p.join) {
            const unsigned y = (unsigned)std::min(p.tile_tiles, 1 << 15), z = ((unsigned)p.tile_tiles + y - 1) / y;
            attention_join_kernel<D><<<dim3((unsigned)(a.Hkv * (M::BM / 16)), y, z), 256, 0, st>>>(c);
        }
    }
    if (p.rows) {
        a.few = p.tiles ? 1 : -1;
        a.items = p.row_items;
        a.target = p.row_target;
        a.least = p.row_least;
        a.stream = p.stream;
        launch(&attention_rows_kernel<D, E4M3>, rows_done, (int64_t)a.items * a.Hkv, R::LDS, a, st);
    }
}

}  // namespace

size_t paged_attention_workspace_bytes(int T, int B, int64_t max_kv, int Hq, int Hkv, int D, int prefix, int max_q) {
    if (T == 0 || B == 0) return 0;
    return std::max(plan_of(T, B, max_kv, Hq, Hkv, D, false, prefix, max_q).bytes(),
                    plan_of(T, B, max_kv, Hq, Hkv, D, true, prefix, max_q).bytes());
}

void launch_paged_attention(const AttentionArgs& args, int D, void* ws, hipStream_t st) {
    Call a{args};
    a.G = a.Hq / a.Hkv;
    a.scale2 = a.scale * kLog2E;
    a.shared = a.prefix;
    const Plan p = plan_of(a.T, a.B, (int64_t)a.max_pages << a.page_shift, a.Hq, a.Hkv, D, a.k_scale != nullptr, a.prefix, a.max_q);
    if (!p.prior_chunks) a.prefix = 0;                   // every sequence reads the shared pages for itself
    if (D == 64) a.k_scale ? launch_all<64, true>(a, p, ws, st) : launch_all<64, false>(a, p, ws, st);
    else a.k_scale ? launch_all<128, true>(a, p, ws, st) : launch_all<128, false>(a, p, ws, st);
}

}  // namespace qg
