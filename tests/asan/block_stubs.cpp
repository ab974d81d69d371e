// Host-only stand-ins for the launchers behind abi_block.cpp (test
// infrastructure): they record each call and touch no memory.
#include <hip/hip_runtime.h>

#include "launch.h"

int g_launches = 0;

namespace qg {

void launch_rms_norm(const uint16_t*, const uint16_t*, const uint16_t*, float, int, int, uint16_t*, uint16_t*, void*,
                     float*, ActFormat, hipStream_t) { ++g_launches; }
void launch_swiglu(const uint16_t*, int, int, uint16_t*, void*, float*, ActFormat, hipStream_t) { ++g_launches; }
size_t w4a16_workspace_bytes(int M, int, int) { return M > 64 ? 4096 : 0; }
void launch_qgemm_w4a16_epilogue(const uint16_t*, const uint32_t*, const uint16_t*, const uint16_t*, int,
                                 const uint16_t*, uint16_t*, int, int, int, void*, hipStream_t) { ++g_launches; }
size_t moe_dispatch_workspace_bytes(int B, int k, int E) { return B * k > 64 ? (size_t)E * 4 : 0; }
void launch_moe_dispatch(const int*, const void*, const float*, int, int, int, int, int*, int*, void*, float*, void*,
                         hipStream_t) { ++g_launches; }
void launch_moe_gather(const void*, const float*, const int*, int, int, int, void*, float*, hipStream_t) { ++g_launches; }
void launch_moe_combine(const uint16_t*, const int*, const float*, const uint16_t*, int, int, int, uint16_t*,
                        hipStream_t) { ++g_launches; }
void launch_moe_combine_backward(const uint16_t*, const uint16_t*, const int*, const float*, int, int, int, uint16_t*,
                                 float*, hipStream_t) { ++g_launches; }

}  // namespace qg
