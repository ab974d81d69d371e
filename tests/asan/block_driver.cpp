// Exercises the entry points of abi_block.cpp with stub launchers (test
// infrastructure, host only): invalid arguments return their status without
// launching, valid ones reach the launcher once.  Prints "abi block driver ok".
#include <climits>
#include <cstdio>
#include <initializer_list>

#include "../../include/qgemm.h"

extern int g_launches;

static int failures = 0;
static void expect(int line, int launched, bool status_ok, int want) {
    if (!status_ok || launched != want) {
        std::fprintf(stderr, "line %d: status %s, %d launches\n", line, status_ok ? "as expected" : "wrong", launched);
        ++failures;
    }
}
// a launch without a GPU reports OK or HIP
#define LAUNCHES(call)                                                                \
    do {                                                                              \
        const int before = g_launches;                                                \
        const qg_status st = (call);                                                  \
        expect(__LINE__, g_launches - before, st == QG_OK || st == QG_ERR_HIP, 1);    \
    } while (0)
#define REFUSED(call, want)                                                           \
    do {                                                                              \
        const int before = g_launches;                                                \
        const qg_status st = (call);                                                  \
        expect(__LINE__, g_launches - before, st == (want), 0);                       \
    } while (0)

alignas(256) static unsigned char mem[4096];

int main() {
    auto* h = reinterpret_cast<uint16_t*>(mem);
    auto* f = reinterpret_cast<float*>(mem);
    auto* i = reinterpret_cast<int32_t*>(mem);
    auto* w = reinterpret_cast<uint32_t*>(mem);
    auto* b = reinterpret_cast<uint8_t*>(mem);
    auto* s = reinterpret_cast<int8_t*>(mem);

    LAUNCHES(rms_norm(h, nullptr, h, 1e-5f, 3, 64, nullptr, h, nullptr));
    LAUNCHES(rms_norm_quant(h, h, h, 1e-5f, 3, 64, h, nullptr, b, f, nullptr));
    LAUNCHES(rms_norm_quant_int8(h, h, h, 1e-5f, 3, 64, h, h, s, f, nullptr));
    REFUSED(rms_norm(h, nullptr, h, 1e-5f, INT_MAX, INT_MAX, nullptr, h, nullptr), QG_ERR_SHAPE);
    REFUSED(rms_norm(h, nullptr, h, 1e-5f, INT_MIN, 64, nullptr, h, nullptr), QG_ERR_SHAPE);
    REFUSED(rms_norm(h, nullptr, h, 0.0f, 3, 64, nullptr, h, nullptr), QG_ERR_SHAPE);
    REFUSED(rms_norm_quant(h, h, h, 1e-5f, 3, 64, h, nullptr, nullptr, f, nullptr), QG_ERR_NULL);
    REFUSED(rms_norm_quant_int8(h, h, h, 1e-5f, 3, 64, h, h, s + 8, f, nullptr), QG_ERR_ALIGN);
    LAUNCHES(swiglu(h, 3, 64, h, nullptr));
    LAUNCHES(swiglu_quant(h, 3, 64, b, f, nullptr));
    LAUNCHES(swiglu_quant_int8(h, 3, 64, s, f, nullptr));
    REFUSED(swiglu(h, 3, INT_MAX, h, nullptr), QG_ERR_SHAPE);
    REFUSED(swiglu_quant(h + 1, 3, 64, b, f, nullptr), QG_ERR_ALIGN);

    LAUNCHES(qgemm_w4a16_epilogue(h, w, h, h, QG_ACT_GELU, h, h, 4, 64, 256, nullptr, 0, nullptr));
    LAUNCHES(qgemm_w4a16_epilogue(h, w, h, nullptr, QG_ACT_NONE, nullptr, h, 100, 64, 256, mem, 4096, nullptr));
    REFUSED(qgemm_w4a16_epilogue(h, w, h, h, QG_ACT_GELU, h, h, 100, 64, 256, mem, 4095, nullptr), QG_ERR_WORKSPACE);
    REFUSED(qgemm_w4a16_epilogue(h, w, h, h, INT_MAX, h, h, 4, 64, 256, nullptr, 0, nullptr), QG_ERR_SHAPE);
    REFUSED(qgemm_w4a16_epilogue(h, w, h, h, QG_ACT_SILU, h + 1, h, 4, 64, 256, nullptr, 0, nullptr), QG_ERR_ALIGN);

    LAUNCHES(moe_dispatch(i, mem, f, 4, 8, 128, 64, i, i, mem, f, nullptr, 0, nullptr));
    LAUNCHES(moe_dispatch(i, nullptr, nullptr, 4, 8, 128, INT_MIN, i, i, nullptr, nullptr, nullptr, 0, nullptr));
    LAUNCHES(moe_dispatch(nullptr, nullptr, nullptr, 0, 8, 128, 0, i, nullptr, nullptr, nullptr, nullptr, 0, nullptr));
    LAUNCHES(moe_dispatch(i, mem, f, 400, 8, 128, 64, i, i, mem, f, mem, 512, nullptr));
    REFUSED(moe_dispatch(i, mem, f, 400, 8, 128, 64, i, i, mem, f, mem, 511, nullptr), QG_ERR_WORKSPACE);
    REFUSED(moe_dispatch(i, mem, f, INT_MAX, INT_MAX, 128, 64, i, i, mem, f, mem, 512, nullptr), QG_ERR_SHAPE);
    REFUSED(moe_dispatch(i, mem, f, 4, 8, INT_MAX, 64, i, i, mem, f, mem, 512, nullptr), QG_ERR_SHAPE);
    REFUSED(moe_dispatch(i, mem, f, 4, 8, 128, INT_MAX - 7, i, i, mem, f, mem, 512, nullptr), QG_ERR_SHAPE);
    LAUNCHES(moe_gather(mem, nullptr, i, 4, 8, 64, mem, nullptr, nullptr));
    REFUSED(moe_gather(mem, f, i, 4, 8, 64, mem, nullptr, nullptr), QG_ERR_NULL);
    REFUSED(moe_gather(mem, nullptr, i, 0, 8, 64, mem, nullptr, nullptr), QG_OK);
    LAUNCHES(moe_combine(h, i, nullptr, nullptr, 4, 8, 64, h, nullptr));
    REFUSED(moe_combine(h, i, f, h, 4, 8, INT_MAX - 7, h, nullptr), QG_ERR_SHAPE);
    LAUNCHES(moe_combine_backward(h, h, i, f, 4, 8, 64, h, f, nullptr));
    LAUNCHES(moe_combine_backward(h, nullptr, i, f, 4, 8, 64, h, nullptr, nullptr));
    REFUSED(moe_combine_backward(h, nullptr, i, f, 4, 8, 64, h, f, nullptr), QG_ERR_NULL);

    for (int64_t B : {int64_t(-1), int64_t(0), int64_t(1), int64_t(1) << 24, INT64_MAX})
        for (int64_t k : {int64_t(-1), int64_t(0), int64_t(1), int64_t(1024), INT64_MAX})
            for (int64_t E : {int64_t(0), int64_t(1), int64_t(1024), INT64_MAX})
                (void)qg_moe_dispatch_workspace_bytes(B, k, E);

    if (failures) return 1;
    std::puts("abi block driver ok");
    return 0;
}
