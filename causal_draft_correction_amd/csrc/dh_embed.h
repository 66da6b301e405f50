// Embedding rows and the table's gradient: launches of the device code in domino_embed.hip.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/domino_head.h"

namespace dhembed {

// Arguments were checked by the caller.
hipError_t forward(const domino_rows &table, const int32_t *ids, float scale, const domino_rows &out, hipStream_t st);

size_t workspace_bytes(const domino_rows &grad);
// accumulate: rows of `table` that tokens name are added to, the others left; else all of it is written.
hipError_t backward(const domino_rows &grad, const int32_t *ids, float scale, bool accumulate, void *ws,
                    const domino_rows &table, hipStream_t st);

}  // namespace dhembed
