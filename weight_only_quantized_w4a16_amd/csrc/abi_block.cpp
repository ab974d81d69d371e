// C ABI of the operators between the products (declared in include/qgemm.h):
// argument validation on the host, before anything is launched, then dispatch.
#include <float.h>
#include <hip/hip_runtime.h>

#include "../../include/qgemm.h"
#include "abi_common.h"
#include "launch.h"

using namespace qg;

namespace {

// Row operators launch up to 1024 threads a row and expert ones 256 a 256-piece
// part of a token's row; a dispatch holds fewer than 2^32 threads.
constexpr int64_t kMaxRows = (int64_t(1) << 22) - 1;
constexpr int64_t kMaxGatedElems = (int64_t(1) << 35) - 2048;
constexpr int64_t kMaxSlots = int64_t(1) << 24;          // routed rows
constexpr int kMaxChoices = 1024;                        // experts of one token

bool rows_ok(int64_t M, int64_t K) {
    return M >= 0 && M <= kMaxRows && K > 0 && K <= kMaxK && K % 8 == 0 && M * K < (int64_t(1) << 35);
}

bool slots_ok(int64_t B, int64_t k) {
    return B >= 0 && B <= kMaxRows && k >= 1 && k <= kMaxChoices && B * k <= kMaxSlots;
}

// the pieces of B rows fit one launch (256 pieces a workgroup at most)
bool token_rows_ok(int64_t B, int64_t pieces) { return B * ((pieces + 255) / 256) < (int64_t(1) << 24); }

bool eps_ok(float eps) { return eps >= FLT_MIN && eps <= FLT_MAX; }   // positive, normal

qg_status norm(const uint16_t* x, const uint16_t* r, const uint16_t* w, float eps, int M, int K, uint16_t* h,
               uint16_t* y, void* q, float* s, ActFormat fmt, qg_stream stream) {
    if (!rows_ok(M, K) || !eps_ok(eps)) return QG_ERR_SHAPE;
    if (M == 0) return QG_OK;
    if (!x || !w) return QG_ERR_NULL;
    if (fmt == ActFormat::bf16 ? !y : !q || !s) return QG_ERR_NULL;
    if (!aligned(x, 16) || !aligned(r, 16) || !aligned(w, 16) || !aligned(h, 16) || !aligned(y, 16) ||
        !aligned(q, 16) || !aligned(s, 4))
        return QG_ERR_ALIGN;
    launch_rms_norm(x, r, w, eps, M, K, h, y, q, s, fmt, as_stream(stream));
    return launched();
}

qg_status gated(const uint16_t* gu, int M, int I, uint16_t* y, void* q, float* s, ActFormat fmt, qg_stream stream) {
    if (!rows_ok(M, I)) return QG_ERR_SHAPE;
    // the bf16 output's launch: a thread per eight elements, 256 a workgroup
    if (fmt == ActFormat::bf16 && int64_t(M) * I > kMaxGatedElems) return QG_ERR_SHAPE;
    if (M == 0) return QG_OK;
    if (!gu || (fmt == ActFormat::bf16 ? !y : !q || !s)) return QG_ERR_NULL;
    if (!aligned(gu, 16) || !aligned(y, 16) || !aligned(q, 16) || !aligned(s, 4)) return QG_ERR_ALIGN;
    launch_swiglu(gu, M, I, y, q, s, fmt, as_stream(stream));
    return launched();
}

}  // namespace

extern "C" {

qg_status rms_norm(const uint16_t* x_bf16, const uint16_t* residual_bf16, const uint16_t* weight_bf16, float eps, int M,
                   int K, uint16_t* h_bf16, uint16_t* y_bf16, qg_stream stream) {
    return norm(x_bf16, residual_bf16, weight_bf16, eps, M, K, h_bf16, y_bf16, nullptr, nullptr, ActFormat::bf16, stream);
}

qg_status rms_norm_quant(const uint16_t* x_bf16, const uint16_t* residual_bf16, const uint16_t* weight_bf16, float eps,
                         int M, int K, uint16_t* h_bf16, uint16_t* y_bf16, uint8_t* y_e4m3, float* y_scale,
                         qg_stream stream) {
    return norm(x_bf16, residual_bf16, weight_bf16, eps, M, K, h_bf16, y_bf16, y_e4m3, y_scale, ActFormat::e4m3, stream);
}

qg_status rms_norm_quant_int8(const uint16_t* x_bf16, const uint16_t* residual_bf16, const uint16_t* weight_bf16,
                              float eps, int M, int K, uint16_t* h_bf16, uint16_t* y_bf16, int8_t* y_i8,
                              float* y_scale, qg_stream stream) {
    return norm(x_bf16, residual_bf16, weight_bf16, eps, M, K, h_bf16, y_bf16, y_i8, y_scale, ActFormat::int8, stream);
}

qg_status swiglu(const uint16_t* gate_up_bf16, int M, int I, uint16_t* y_bf16, qg_stream stream) {
    return gated(gate_up_bf16, M, I, y_bf16, nullptr, nullptr, ActFormat::bf16, stream);
}

qg_status swiglu_quant(const uint16_t* gate_up_bf16, int M, int I, uint8_t* y_e4m3, float* y_scale, qg_stream stream) {
    return gated(gate_up_bf16, M, I, nullptr, y_e4m3, y_scale, ActFormat::e4m3, stream);
}

qg_status swiglu_quant_int8(const uint16_t* gate_up_bf16, int M, int I, int8_t* y_i8, float* y_scale, qg_stream stream) {
    return gated(gate_up_bf16, M, I, nullptr, y_i8, y_scale, ActFormat::int8, stream);
}

qg_status qgemm_w4a16_epilogue(const uint16_t* a_bf16, const uint32_t* packed, const uint16_t* scales,
                               const uint16_t* bias_bf16, int activation, const uint16_t* residual_bf16,
                               uint16_t* y_bf16, int M, int N, int K, void* workspace, size_t workspace_bytes,
                               qg_stream stream) {
    if (!shape_ok(M, N, K) || activation < QG_ACT_NONE || activation > QG_ACT_SILU) return QG_ERR_SHAPE;
    if (M == 0) return QG_OK;
    if (!a_bf16 || !packed || !scales || !y_bf16) return QG_ERR_NULL;
    if (!aligned(a_bf16, 16) || !aligned(packed, 16) || !aligned(scales, 4) || !aligned(bias_bf16, 4) ||
        !aligned(residual_bf16, 16) || !aligned(y_bf16, 16))
        return QG_ERR_ALIGN;
    const size_t need = w4a16_workspace_bytes(M, N, K);
    if (need > 0) {
        if (!workspace) return QG_ERR_NULL;
        if (workspace_bytes < need) return QG_ERR_WORKSPACE;
        if (!aligned(workspace, 16)) return QG_ERR_ALIGN;
    }
    launch_qgemm_w4a16_epilogue(a_bf16, packed, scales, bias_bf16, activation, residual_bf16, y_bf16, M, N, K, workspace,
                                as_stream(stream));
    return launched();
}

// ---- expert routing ----

size_t qg_moe_dispatch_workspace_bytes(int64_t B, int64_t k, int64_t E) {
    if (!slots_ok(B, k) || E < 1 || E > kGroupedMaxExperts) return 0;
    return moe_dispatch_workspace_bytes((int)B, (int)k, (int)E);
}

qg_status moe_dispatch(const int32_t* expert_ids, const void* rows, const float* row_scale, int B, int k, int E,
                       int row_bytes, int32_t* offsets, int32_t* row_of_slot, void* rows_out, float* row_scale_out,
                       void* workspace, size_t workspace_bytes, qg_stream stream) {
    if (!slots_ok(B, k) || E < 1 || E > kGroupedMaxExperts) return QG_ERR_SHAPE;
    if (rows && (row_bytes <= 0 || row_bytes % 8 != 0 || row_bytes > 2 * kMaxK || !token_rows_ok(B, row_bytes / 8)))
        return QG_ERR_SHAPE;
    if (!offsets) return QG_ERR_NULL;
    if (B > 0 && (!expert_ids || !row_of_slot || !rows != !rows_out || !row_scale != !row_scale_out ||
                  (row_scale && !rows)))
        return QG_ERR_NULL;
    if (!aligned(expert_ids, 4) || !aligned(rows, 16) || !aligned(row_scale, 4) || !aligned(offsets, 4) ||
        !aligned(row_of_slot, 4) || !aligned(rows_out, 16) || !aligned(row_scale_out, 4))
        return QG_ERR_ALIGN;
    const size_t need = moe_dispatch_workspace_bytes(B, k, E);
    if (need > 0) {
        if (!workspace) return QG_ERR_NULL;
        if (workspace_bytes < need) return QG_ERR_WORKSPACE;
        if (!aligned(workspace, 4)) return QG_ERR_ALIGN;
    }
    launch_moe_dispatch(expert_ids, rows, row_scale, B, k, E, row_bytes, offsets, row_of_slot, rows_out, row_scale_out,
                        workspace, as_stream(stream));
    return launched();
}

qg_status moe_gather(const void* rows, const float* row_scale, const int32_t* row_of_slot, int B, int k, int row_bytes,
                     void* rows_out, float* row_scale_out, qg_stream stream) {
    if (!slots_ok(B, k) || row_bytes <= 0 || row_bytes % 8 != 0 || row_bytes > 2 * kMaxK ||
        !token_rows_ok(B, row_bytes / 8))
        return QG_ERR_SHAPE;
    if (B == 0) return QG_OK;
    if (!rows || !row_of_slot || !rows_out || !row_scale != !row_scale_out) return QG_ERR_NULL;
    if (!aligned(rows, 16) || !aligned(row_scale, 4) || !aligned(row_of_slot, 4) || !aligned(rows_out, 16) ||
        !aligned(row_scale_out, 4))
        return QG_ERR_ALIGN;
    launch_moe_gather(rows, row_scale, row_of_slot, B, k, row_bytes, rows_out, row_scale_out, as_stream(stream));
    return launched();
}

qg_status moe_combine(const uint16_t* rows_bf16, const int32_t* row_of_slot, const float* weights,
                      const uint16_t* residual_bf16, int B, int k, int K, uint16_t* y_bf16, qg_stream stream) {
    if (!slots_ok(B, k) || K <= 0 || K % 8 != 0 || K > kMaxK || !token_rows_ok(B, K / 8)) return QG_ERR_SHAPE;
    if (B == 0) return QG_OK;
    if (!rows_bf16 || !row_of_slot || !y_bf16) return QG_ERR_NULL;
    if (!aligned(rows_bf16, 16) || !aligned(row_of_slot, 4) || !aligned(weights, 4) || !aligned(residual_bf16, 16) ||
        !aligned(y_bf16, 16))
        return QG_ERR_ALIGN;
    launch_moe_combine(rows_bf16, row_of_slot, weights, residual_bf16, B, k, K, y_bf16, as_stream(stream));
    return launched();
}

qg_status moe_combine_backward(const uint16_t* dy_bf16, const uint16_t* rows_bf16, const int32_t* row_of_slot,
                               const float* weights, int B, int k, int K, uint16_t* drows_bf16, float* dweights,
                               qg_stream stream) {
    if (!slots_ok(B, k) || K <= 0 || K % 8 != 0 || K > kMaxK || !token_rows_ok(B, K / 8)) return QG_ERR_SHAPE;
    if (B == 0) return QG_OK;
    if (!dy_bf16 || !row_of_slot || (!drows_bf16 && !dweights) || (dweights && !rows_bf16)) return QG_ERR_NULL;
    if (!aligned(dy_bf16, 16) || !aligned(rows_bf16, 16) || !aligned(row_of_slot, 4) || !aligned(weights, 4) ||
        !aligned(drows_bf16, 16) || !aligned(dweights, 4))
        return QG_ERR_ALIGN;
    launch_moe_combine_backward(dy_bf16, rows_bf16, row_of_slot, weights, B, k, K, drows_bf16, dweights,
                                as_stream(stream));
    return launched();
}

}  // extern "C"
