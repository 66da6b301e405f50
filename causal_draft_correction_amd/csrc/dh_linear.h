// Linear layers and their gradients: launches of the device code in domino_linear.hip and domino_linear_*.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/domino_head.h"

namespace dhlinear {

// Tiles of a product: 128 x 128, 64 x 64, 64 x 16 (forward), 256 x 256 (two bfloat16 operands).
enum Shape { LARGE, MEDIUM, FEW, HUGE };

struct Forward {
    const domino_rows *x, *weight, *bias, *residual, *y, *pre;  // bias, residual, pre: NULL for none
    int act;
};
struct Backward {
    const domino_rows *grad, *x, *weight, *pre;  // pre: NULL without an activation
    const domino_rows *grad_x, *grad_weight, *grad_bias;  // NULL: not wanted
    int act;
    bool accumulate;
};

// Arguments were checked by the caller.  (Workspaces go by sizes, and by which gradients there are.)
size_t workspace_bytes(const Forward &f);
hipError_t forward(const Forward &f, void *ws, hipStream_t st);
size_t workspace_bytes(const Backward &b);
hipError_t backward(const Backward &b, void *ws, hipStream_t st);

}  // namespace dhlinear
