// logprobs.h -- launcher of the log-probability kernels (logprobs.hip).
#pragma once

#include "qlinear_internal.h"

namespace ql {

struct LogprobArgs {
    const float *logits;   // [M] rows of V, ld apart
    int64_t M, V, ld;
    const int32_t *targets;  // [M] or null
    int top;
    float *logprob;        // [M] or null
    int32_t *rank;         // [M] or null
    float *entropy;        // [M] or null
    int32_t *top_ids;      // [M][top] or null when top == 0
    float *top_logprobs;
    uint8_t *ws;
};

// Bytes of one call, and the most that a call with up to M rows and up to `top`
// alternatives needs.
int64_t logprobs_need(int64_t M, int64_t V, int top);
int64_t logprobs_workspace(int64_t M, int64_t V, int top);

hipError_t launch_logprobs(const LogprobArgs &a, hipStream_t s);

}  // namespace ql
