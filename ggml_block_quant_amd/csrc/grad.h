// grad.h -- launchers of the gradients through frozen quantized weights and of
// the head's cross entropy (grad.hip).
#pragma once

#include "qlinear_internal.h"

namespace ql {

// dX [M][K] (bf16) = dY [M][N] . deq(W)
struct GradArgs {
    int fmt;
    const uint8_t *W;
    const void *dY;
    bool dy_bf16;   // else fp32
    uint16_t *dX;
    int64_t M, N, K;
    uint8_t *ws;
};
int64_t grad_workspace(int fmt, int64_t M, int64_t N, int64_t K);
hipError_t launch_grad(const GradArgs &a, hipStream_t s);

// The gated pair: dX [M][K] and, where wanted, dG and dU [M][F], all bf16
struct GluGradArgs {
    int fmt, act;
    const uint8_t *gate, *up;
    const uint16_t *X;   // bf16 [M][K]
    const void *dH;      // [M][F]
    bool dh_bf16;
    uint16_t *dX, *dG, *dU;
    int64_t M, F, K;
    uint8_t *ws;
};
int64_t glu_grad_workspace(int fmt, int64_t M, int64_t F, int64_t K);
hipError_t launch_glu_grad(const GluGradArgs &a, hipStream_t s);

// Cross entropy over the head [N][K]: loss, lse (or null) [M], dX (or null)
struct XentArgs {
    int fmt;
    const uint8_t *W;
    const uint16_t *X;
    const int32_t *targets;
    const float *weights;   // [M] or null
    float *loss, *lse;
    uint16_t *dX;
    int64_t M, N, K;
    uint8_t *ws;
};
int64_t xent_workspace(int fmt, int64_t M, int64_t N, int64_t K, bool grad);
hipError_t launch_xent(const XentArgs &a, hipStream_t s);

}  // namespace ql
