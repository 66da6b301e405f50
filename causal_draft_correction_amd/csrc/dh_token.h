// Log-probabilities of given tokens, entropies and alternatives: launches of the device code in domino_token.hip (and, for
// alternatives, domino_top.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/domino_head.h"

namespace dhtoken {

constexpr int STATS = 8;  // floats of a row's statistics

struct Scores {
    const int32_t *tokens;       // [B, R]
    float *logprob, *entropy;    // [B, R]
    float *stats;                // [B, R, STATS] or NULL
};

size_t workspace_bytes(const domino_logits &lg);
// Arguments were checked by the caller.
hipError_t forward(const domino_logits &lg, const Scores &s, double tau, const int32_t *n_rows, void *ws,
                   hipStream_t st);
// grad_logprob or grad_entropy may be NULL: 0.
hipError_t both(const domino_logits &lg, const Scores &s, double tau, const int32_t *n_rows, void *ws,
                const float *grad_logprob, const float *grad_entropy, const domino_logits &grad, hipStream_t st);
hipError_t backward(const domino_logits &lg, const int32_t *tokens, const float *stats, const float *grad_logprob,
                    const float *grad_entropy, double tau, const int32_t *n_rows, const domino_logits &grad,
                    hipStream_t st);

}  // namespace dhtoken
