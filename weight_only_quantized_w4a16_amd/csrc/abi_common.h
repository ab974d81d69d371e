// Argument checks shared by the C-ABI files.
#pragma once

#include <hip/hip_runtime.h>

#include "../../include/qgemm.h"

namespace qg {

// Limits that keep every index the kernels form inside its integer type.
constexpr int64_t kMaxDim = int64_t(1) << 24;        // M, N
constexpr int64_t kMaxK = int64_t(1) << 20;          // K
constexpr int64_t kMaxElems = int64_t(1) << 38;      // elements of one matrix

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// K % 128, N % 16, bounds.  M may be 0.
inline bool shape_ok(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N <= 0 || K <= 0) return false;
    if (K % 128 != 0 || N % 16 != 0) return false;
    if (M > kMaxDim || N > kMaxDim || K > kMaxK) return false;
    if (N * K > kMaxElems || M * K > kMaxElems || M * N > kMaxElems) return false;
    return true;
}

inline qg_status launched() {
    return hipGetLastError() == hipSuccess ? QG_OK : QG_ERR_HIP;
}

inline hipStream_t as_stream(qg_stream s) { return reinterpret_cast<hipStream_t>(s); }

}  // namespace qg
