// Launches of the mixture-of-experts layer for a few tokens (moe.hip).  Arguments were
// validated by the API layer.
#pragma once

#include "common.hpp"

namespace convrot {

constexpr int kMoeMaxExperts = 512, kMoeMaxShared = 16, kMoeMaxTopK = 32;
constexpr int kMoeTokens = 64;             // tokens of one pass over the experts

// One pass: T <= kMoeTokens tokens.
struct Moe {
    const uint16_t *x;                     // bf16 [T, K]
    const void *router;                    // [E, K], bf16 or fp32
    const float *bias;                     // [E] or null
    const uint8_t *gate_up, *down;         // E + S experts of [2F, K] and [K, F], K-tiled codes
    const float *gate_up_scale, *down_scale;
    int T, E, S, top_k, K, F;
    bool router_f32, sigmoid, renormalize, y_f32;
    double factor;
    void *y;                               // [T, K]
    int32_t *ids;                          // [T, top_k]
    float *weights;
    void *ws;                              // moe_workspace_bytes
};
// For passes of up to T tokens.
size_t moe_workspace_bytes(int T, int E, int S, int top_k, int K, int F);
// Whether gate_up chooses the experts itself, in a launch of so many workgroups.
bool moe_own_choice(int T, int64_t workgroups, int64_t cus);
hipError_t launch_moe(const Moe &m, hipStream_t stream);

} // namespace convrot
