// moe.h -- launchers of the mixture-of-experts kernels (moe.hip).
#pragma once

#include "qlinear_internal.h"

namespace ql {

// Shapes of one mixture-of-experts call.  gate / up: [E*F][K] in fmt_gu,
// down: [E*K][F] in fmt_d (the experts' tensors stacked along the rows).
struct MoeArgs {
    int fmt_gu, fmt_d, act;
    int T, E, k;      // tokens, experts, experts per token
    int64_t F, K;     // inner width of an expert, model width
    const uint8_t *gate, *up, *down;
    const uint16_t *X;      // bf16 [T][K]
    const int32_t *ids;     // [T][k]; outside [0, E): no expert
    const float *weights;   // [T][k]
    float *Y;               // [T][K]
    uint8_t *ws;
};

// Workspace bytes of a call (both forms; see moe.hip for the layout).
int64_t moe_workspace(int T, int E, int k, int64_t F, int64_t K);

hipError_t launch_moe(const MoeArgs &a, hipStream_t s);

hipError_t launch_moe_route(const float *logits, int T, int E, int k, int score, const float *bias, int renorm,
                            float scale, int32_t *ids, float *weights, hipStream_t s);

}  // namespace ql
