// C ABI of the operators between the qkv product and the o product (declared in
// include/qgemm.h): argument validation on the host, before anything is launched,
// then dispatch.
#include <float.h>
#include <hip/hip_runtime.h>
#include <math.h>

#include "../../include/qgemm.h"
#include "abi_common.h"
#include "launch.h"

using namespace qg;

namespace {

// Every thread of a launch and every index a kernel forms fit their types: a wave a
// token, a workgroup a work item, of which there are at most T Hq / 16 + B Hkv + those
// of the keys' chunks.
constexpr int64_t kMaxTokens = (int64_t(1) << 22) - 1;
constexpr int kMaxHeads = 1024;
constexpr int64_t kMaxQueryRows = int64_t(1) << 27;      // T Hq
constexpr int kMaxSequences = 1 << 14;
constexpr int64_t kMaxPositions = int64_t(1) << 30;      // of a sequence
constexpr int64_t kMaxCacheRows = int64_t(1) << 40;      // pages Hkv page

bool heads_ok(int64_t T, int64_t Hq, int64_t Hkv, int64_t D) {
    return T >= 0 && T <= kMaxTokens && Hkv >= 1 && Hq >= Hkv && Hq <= kMaxHeads && Hq % Hkv == 0 &&
           (D == 64 || D == 128) && T * Hq <= kMaxQueryRows;
}

int page_shift(int64_t page) {
    for (int s = 4; s <= 8; ++s)
        if (page == int64_t(1) << s) return s;
    return -1;
}

bool batch_ok(int64_t B, int64_t max_pages, int64_t page, int64_t Hkv) {
    return B >= 0 && B <= kMaxSequences && B * Hkv < (int64_t(1) << 23) && max_pages >= 1 &&
           max_pages <= kMaxPositions && page_shift(page) > 0 && max_pages * page <= kMaxPositions;
}

bool cache_ok(int64_t pages, int64_t page, int64_t Hkv) { return pages >= 1 && pages * page * Hkv <= kMaxCacheRows; }

// rotation and norm of a call
bool rope_ok(float eps, bool norm, int rot, int D) {
    return rot >= 0 && rot <= D && rot % 16 == 0 && (!norm || (eps >= FLT_MIN && eps <= FLT_MAX));
}

}  // namespace

extern "C" {

qg_status qk_norm_rope(const uint16_t* qkv_bf16, const uint16_t* q_weight_bf16, const uint16_t* k_weight_bf16, float eps,
                       const int32_t* positions, const double* inv_freq, int rotary_dim, int interleaved, int T, int Hq,
                       int Hkv, int D, uint16_t* q_bf16, uint16_t* k_bf16, qg_stream stream) {
    if (!heads_ok(T, Hq, Hkv, D) || !rope_ok(eps, q_weight_bf16 || k_weight_bf16, rotary_dim, D)) return QG_ERR_SHAPE;
    if (T == 0) return QG_OK;
    if (!qkv_bf16 || !positions || !q_bf16 || !k_bf16 || (rotary_dim > 0 && !inv_freq)) return QG_ERR_NULL;
    if (!aligned(qkv_bf16, 16) || !aligned(q_weight_bf16, 16) || !aligned(k_weight_bf16, 16) || !aligned(positions, 4) ||
        !aligned(inv_freq, 8) || !aligned(q_bf16, 16) || !aligned(k_bf16, 16))
        return QG_ERR_ALIGN;
    RopeArgs p{};
    p.qkv = qkv_bf16;
    p.wq = q_weight_bf16;
    p.wk = k_weight_bf16;
    p.eps = eps;
    p.inv_freq = inv_freq;
    p.rot = rotary_dim;
    p.interleaved = interleaved != 0;
    p.T = T;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.q = q_bf16;
    p.positions = positions;
    p.k_dense = k_bf16;
    launch_qk_norm_rope(p, D, as_stream(stream));
    return launched();
}

qg_status kv_append(const uint16_t* qkv_bf16, const uint16_t* q_weight_bf16, const uint16_t* k_weight_bf16, float eps,
                    const double* inv_freq, int rotary_dim, int interleaved, const int32_t* q_offsets,
                    const int32_t* kv_len, const int32_t* block_table, int T, int B, int max_pages, int Hq, int Hkv, int D,
                    void* k_cache, void* v_cache, float* k_scale, float* v_scale, int pages, int page_size,
                    uint16_t* q_bf16, qg_stream stream) {
    if (!heads_ok(T, Hq, Hkv, D) || !batch_ok(B, max_pages, page_size, Hkv) || !cache_ok(pages, page_size, Hkv) ||
        !rope_ok(eps, q_weight_bf16 || k_weight_bf16, rotary_dim, D))
        return QG_ERR_SHAPE;
    if (T == 0 || B == 0) return QG_OK;
    if (!qkv_bf16 || !q_offsets || !kv_len || !block_table || !k_cache || !v_cache || !k_scale != !v_scale || !q_bf16 ||
        (rotary_dim > 0 && !inv_freq))
        return QG_ERR_NULL;
    if (!aligned(qkv_bf16, 16) || !aligned(q_weight_bf16, 16) || !aligned(k_weight_bf16, 16) || !aligned(inv_freq, 8) ||
        !aligned(q_offsets, 4) || !aligned(kv_len, 4) || !aligned(block_table, 4) || !aligned(k_cache, 16) ||
        !aligned(v_cache, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(q_bf16, 16))
        return QG_ERR_ALIGN;
    RopeArgs p{};
    p.qkv = qkv_bf16;
    p.wq = q_weight_bf16;
    p.wk = k_weight_bf16;
    p.eps = eps;
    p.inv_freq = inv_freq;
    p.rot = rotary_dim;
    p.interleaved = interleaved != 0;
    p.T = T;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.q = q_bf16;
    p.q_offsets = q_offsets;
    p.kv_len = kv_len;
    p.table = block_table;
    p.B = B;
    p.max_pages = max_pages;
    p.pages = pages;
    p.page_shift = page_shift(page_size);
    p.k = k_cache;
    p.v = v_cache;
    p.k_scale = k_scale;
    p.v_scale = v_scale;
    launch_kv_append(p, D, as_stream(stream));
    return launched();
}

size_t qg_paged_attention_workspace_bytes(int64_t T, int64_t B, int64_t max_pages, int64_t Hq, int64_t Hkv, int64_t D,
                                          int64_t page_size, int64_t shared_prefix, int64_t max_q) {
    if (!heads_ok(T, Hq, Hkv, D) || !batch_ok(B, max_pages, page_size, Hkv) || shared_prefix < 0 ||
        shared_prefix % page_size != 0 || shared_prefix > max_pages * page_size || max_q < 0)
        return 0;
    return paged_attention_workspace_bytes((int)T, (int)B, max_pages * page_size, (int)Hq, (int)Hkv, (int)D,
                                           (int)shared_prefix, (int)(max_q < T ? max_q : T));
}

qg_status paged_attention(const uint16_t* q_bf16, const void* k_cache, const void* v_cache, const float* k_scale,
                          const float* v_scale, int pages, int page_size, const int32_t* q_offsets, const int32_t* kv_len,
                          const int32_t* block_table, int T, int B, int max_pages, int Hq, int Hkv, int D, float scale,
                          int window, int sinks, int shared_prefix, int max_q, uint16_t* out_bf16, float* lse,
                          void* workspace, size_t workspace_bytes, qg_stream stream) {
    if (!heads_ok(T, Hq, Hkv, D) || !batch_ok(B, max_pages, page_size, Hkv) || !cache_ok(pages, page_size, Hkv) ||
        !isfinite(scale * kLog2E) || window < 0 || window > kMaxPositions || sinks < 0 || max_q < 0 || shared_prefix < 0 ||
        shared_prefix % page_size != 0 || shared_prefix > (int64_t)max_pages * page_size)
        return QG_ERR_SHAPE;
    if (T == 0 || B == 0) return QG_OK;
    if (!q_bf16 || !k_cache || !v_cache || !k_scale != !v_scale || !q_offsets || !kv_len || !block_table || !out_bf16)
        return QG_ERR_NULL;
    if (!aligned(q_bf16, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(k_scale, 4) ||
        !aligned(v_scale, 4) || !aligned(q_offsets, 4) || !aligned(kv_len, 4) || !aligned(block_table, 4) ||
        !aligned(out_bf16, 16) || !aligned(lse, 4))
        return QG_ERR_ALIGN;
    const int most = max_q < T ? max_q : T;
    const size_t need =
        paged_attention_workspace_bytes(T, B, (int64_t)max_pages * page_size, Hq, Hkv, D, shared_prefix, most);
    if (need > 0) {
        if (!workspace) return QG_ERR_NULL;
        if (workspace_bytes < need) return QG_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return QG_ERR_ALIGN;
    }
    AttentionArgs a{};
    a.q = q_bf16;
    a.k = k_cache;
    a.v = v_cache;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.q_offsets = q_offsets;
    a.kv_len = kv_len;
    a.table = block_table;
    a.T = T;
    a.B = B;
    a.max_pages = max_pages;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.pages = pages;
    a.page_shift = page_shift(page_size);
    a.scale = scale;
    a.window = window;
    a.sinks = sinks;
    a.prefix = shared_prefix;
    a.max_q = most;
    a.out = out_bf16;
    a.lse = lse;
    launch_paged_attention(a, D, workspace, as_stream(stream));
    return launched();
}

}  // extern "C"
