// The sequences of a batch, as the attention operators receive them: tokens side by
// side, sequence b owning tokens q_offsets[b] .. q_offsets[b + 1] - 1 and, after its
// new tokens, kv_len[b] positions of which the new ones are the last.  Nothing here
// trusts the lists: offsets are clamped into the tokens, lengths to zero and above,
// and a position without a valid page holds no key.
#pragma once

#include "device_common.h"
#include "rows.h"

namespace qg {

struct Sequence {
    int first_token, tokens;     // within the call's T tokens
    int len;                     // positions, the new tokens' included
};

__device__ __forceinline__ Sequence sequence_of(int lo, int hi, int len, int T) {
    Sequence s;
    s.first_token = min(max(lo, 0), T);
    s.tokens = min(max(hi, s.first_token), T) - s.first_token;
    s.len = max(len, 0);
    return s;
}

// The sequence of token t, found by a whole wave: the last of the ascending offsets
// that is not above t (64 of them a step), or -1 if t belongs to none.
__device__ __forceinline__ int sequence_of_token(const int* __restrict__ q_offsets, int B, int t) {
    const int lane = threadIdx.x & 63;
    int below = 0;
    for (int j = 0; j <= B; j += 64) {
        const int o = q_offsets[min(j + lane, B)];
        below += __builtin_popcountll(__ballot(j + lane <= B && o <= t));
    }
    return below >= 1 && below <= B ? below - 1 : -1;
}

// Inclusive prefix sum over the wave's lanes.
__device__ __forceinline__ int wave_scan(int v) {
    v += (int)dpp_u32<0x111>(0u, (uint32_t)v);
    v += (int)dpp_u32<0x112>(0u, (uint32_t)v);
    v += (int)dpp_u32<0x114>(0u, (uint32_t)v);
    v += (int)dpp_u32<0x118>(0u, (uint32_t)v);
    v += (int)dpp_u32<0x142, 0xa>(0u, (uint32_t)v);
    v += (int)dpp_u32<0x143, 0xc>(0u, (uint32_t)v);
    return v;
}

}  // namespace qg
