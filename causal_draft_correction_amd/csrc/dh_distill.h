// Distillation from a teacher's top logits: launches of the device code in domino_distill.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/domino_head.h"

namespace dhdistill {

constexpr int MAX_K = 128;  // teacher logits of a row
constexpr int STAT_HEAD = 4;  // floats of a row's statistics before those of its k ids

// Bytes of scratch: the chunks' parts, and the rows' statistics where the caller does not keep them; none for rows
// that one block takes whole.
size_t workspace_bytes(const domino_logits &lg, int k);

struct Teacher {
    int k;
    const int32_t *ids;    // [B, R, k]
    const float *values;   // [B, R, k]
    const float *lse;      // [B, R] or NULL
};

// Arguments were checked by the caller.
hipError_t forward(const domino_logits &lg, const Teacher &t, double tau, const int32_t *n_rows, void *ws, float *loss,
                   float *stats, hipStream_t st);
hipError_t both(const domino_logits &lg, const Teacher &t, double tau, const int32_t *n_rows, void *ws, float *loss,
                const float *grad_loss, const domino_logits &grad, hipStream_t st);
hipError_t backward(const domino_logits &lg, int k, const int32_t *ids, const float *stats, const float *grad_loss,
                    double tau, const int32_t *n_rows, const domino_logits &grad, hipStream_t st);

}  // namespace dhdistill
