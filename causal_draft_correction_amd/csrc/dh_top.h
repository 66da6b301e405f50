// Top logits and beam selection: launches of the device code in domino_top.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/domino_head.h"
#include "dh_token.h"

namespace dhtop {

constexpr int MAX_K = 128;         // logits kept of a row, continuations of a beam step
constexpr int MAX_W = 32;          // beams
constexpr int MAX_V = 1 << 19;     // longest row: its chunks' candidates have to fit one block's list

// Bytes of scratch for the k largest of each row (k <= V); top() needs none for rows that one block takes whole.
size_t workspace_bytes(const domino_logits &lg, int k, bool for_beams);

// Arguments were checked by the caller.
hipError_t top(const domino_logits &lg, int k, double tau, const int32_t *n_rows, void *ws, int32_t *ids,
               float *values, float *lse, hipStream_t st);
// Token log-probabilities with the k largest of each row as alternatives.
size_t score_workspace_bytes(const domino_logits &lg, int k);
hipError_t scores(const domino_logits &lg, const dhtoken::Scores &want, int k, double tau, const int32_t *n_rows,
                  void *ws, int32_t *ids, float *logprobs, hipStream_t st);
hipError_t beam(const domino_logits &lg, const domino_beam &bm, void *ws, hipStream_t st);

}  // namespace dhtop
