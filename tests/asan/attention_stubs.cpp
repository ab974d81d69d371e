// Host-only stand-ins for the launchers behind abi_attention.cpp (test
// infrastructure): they record each call and touch no memory.
#include <hip/hip_runtime.h>

#include "launch.h"

int g_launches = 0;

namespace qg {

void launch_qk_norm_rope(const RopeArgs&, int, hipStream_t) { ++g_launches; }
void launch_kv_append(const RopeArgs&, int, hipStream_t) { ++g_launches; }
size_t paged_attention_workspace_bytes(int T, int B, int64_t, int, int, int, int, int) { return T * B > 64 ? 4096 : 0; }
void launch_paged_attention(const AttentionArgs&, int, void*, hipStream_t) { ++g_launches; }

}  // namespace qg
