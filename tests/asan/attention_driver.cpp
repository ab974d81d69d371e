// Exercises the entry points of abi_attention.cpp with stub launchers (test
// infrastructure, host only): invalid arguments return their status without
// launching, valid ones reach the launcher once.  Prints "abi attention driver ok".
#include <climits>
#include <cmath>
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

alignas(256) static unsigned char mem[8192];

int main() {
    auto* h = reinterpret_cast<uint16_t*>(mem);
    auto* f = reinterpret_cast<float*>(mem);
    auto* d = reinterpret_cast<double*>(mem);
    auto* i = reinterpret_cast<int32_t*>(mem);

    LAUNCHES(qk_norm_rope(h, h, h, 1e-6f, i, d, 128, 0, 3, 8, 2, 128, h, h, nullptr));
    LAUNCHES(qk_norm_rope(h, nullptr, nullptr, NAN, i, nullptr, 0, 1, 3, 8, 8, 64, h, h, nullptr));
    REFUSED(qk_norm_rope(h, h, h, NAN, i, d, 128, 0, 3, 8, 2, 128, h, h, nullptr), QG_ERR_SHAPE);
    REFUSED(qk_norm_rope(h, h, h, 1e-6f, i, d, INT_MAX, 0, 3, 8, 2, 128, h, h, nullptr), QG_ERR_SHAPE);
    REFUSED(qk_norm_rope(h, h, h, 1e-6f, i, d, INT_MIN, 0, INT_MAX, INT_MAX, INT_MAX, 128, h, h, nullptr), QG_ERR_SHAPE);
    REFUSED(qk_norm_rope(h, h, h, 1e-6f, i, nullptr, 16, 0, 3, 8, 2, 128, h, h, nullptr), QG_ERR_NULL);

    for (float* s : {static_cast<float*>(nullptr), f}) {
        LAUNCHES(kv_append(h, h, h, 1e-6f, d, 64, 0, i, i, i, 3, 2, 4, 8, 2, 64, mem, mem, s, s, 9, 16, h, nullptr));
        LAUNCHES(paged_attention(h, mem, mem, s, s, 9, 16, i, i, i, 3, 2, 4, 8, 2, 64, -0.5f, 5, 2, 32, 1, h, f, nullptr, 0, nullptr));
    }
    REFUSED(kv_append(h, h, h, 1e-6f, d, 64, 0, i, i, i, 3, 2, 4, 8, 2, 64, mem, mem, f, nullptr, 9, 16, h, nullptr), QG_ERR_NULL);
    REFUSED(kv_append(h, h, h, 1e-6f, d, 64, 0, i, i, i, 3, INT_MAX, INT_MAX, 8, 2, 64, mem, mem, f, f, INT_MAX, INT_MAX, h, nullptr), QG_ERR_SHAPE);
    LAUNCHES(paged_attention(h, mem, mem, f, f, INT_MAX, 256, i, i, i, 3, 2, 1 << 22, 8, 2, 64, 0.f, 1 << 30, INT_MAX, 1 << 30, INT_MAX, h, nullptr, nullptr, 0, nullptr));
    LAUNCHES(paged_attention(h, mem, mem, f, f, 9, 16, i, i, i, 65, 2, 4, 8, 2, 64, 0.5f, 0, 0, 0, 0, h, f, mem, 4096, nullptr));
    REFUSED(paged_attention(h, mem, mem, f, f, 9, 16, i, i, i, 65, 2, 4, 8, 2, 64, 0.5f, 0, 0, 0, 0, h, f, mem, 4095, nullptr), QG_ERR_WORKSPACE);
    REFUSED(paged_attention(h, mem, mem, f, f, 9, 16, i, i, i, 3, 2, 4, 8, 2, 64, INFINITY, 0, 0, 0, 0, h, f, nullptr, 0, nullptr), QG_ERR_SHAPE);
    REFUSED(paged_attention(h, mem, mem, f, f, 9, 16, i, i, i, 3, 2, INT_MAX, 8, 2, 64, 0.5f, INT_MIN, INT_MIN, INT_MIN, INT_MIN, h, f, nullptr, 0, nullptr), QG_ERR_SHAPE);
    REFUSED(paged_attention(h, mem, mem, f, f, 9, 16, i, i, i, 3, 2, 4, 8, 2, 64, 0.5f, 0, 0, INT_MAX - 15, 0, h, f, nullptr, 0, nullptr), QG_ERR_SHAPE);
    REFUSED(paged_attention(h, mem, mem, f, f, 9, 16, i, i, i, 0, 2, 4, 8, 2, 64, 0.5f, 0, 0, 0, 0, nullptr, f, nullptr, 0, nullptr), QG_OK);

    for (int64_t T : {int64_t(-1), int64_t(0), int64_t(7), int64_t(1) << 24, INT64_MAX})
        for (int64_t B : {int64_t(-1), int64_t(0), int64_t(3), INT64_MAX})
            for (int64_t w : {int64_t(-1), int64_t(4), int64_t(1) << 40, INT64_MAX})
                for (int64_t n : {int64_t(0), int64_t(8), INT64_MAX, INT64_MIN})
                    (void)qg_paged_attention_workspace_bytes(T, B, w, n, n, 64, n < 0 ? INT64_MIN + 16 : 16, n, n);

    if (failures) return 1;
    std::puts("abi attention driver ok");
    return 0;
}
