// gated.hpp -- the rows of the gated activation.
#pragma once

#include "common.hpp"
#include "launch.hpp"

namespace moe {

// slot of row i: -1 padding, -2 a row past *num_rows (not touched)
__device__ __forceinline__ int gated_slot(const GatedArgs& a, int i) {
    if (a.num_rows && i >= *a.num_rows) return -2;
    if (!a.sorted) return i;
    const uint32_t p = (uint32_t)a.sorted[i];
    return p < a.slots ? (int)p : -1;
}

}  // namespace moe
