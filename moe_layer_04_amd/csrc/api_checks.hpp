// api_checks.hpp -- what the C entry points of the operators around the experts
// share: limits, argument checks and the workspace protocol.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace moe {

constexpr size_t kAlign = 256;
constexpr long kMaxRows = 1L << 28;     // sorted rows, slots
constexpr int kMaxWidth = 1 << 20;      // K, N
constexpr long kMaxThreads = 1L << 32;  // of a launch
constexpr long kMaxGather = 1L << 31;   // bytes of a gathered operand, of one expert's weights

inline bool misaligned(const void* p) { return p && ((uintptr_t)p & 15u); }
inline size_t round_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

// whether two buffers of these many bytes share any
inline bool overlap(const void* p, long np, const void* q, long nq) {
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
    return a < b + (uintptr_t)nq && b < a + (uintptr_t)np;
}

inline moe_status finish() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// workspace == nullptr: reports the size.  Returns true when the call is done.
inline bool workspace_step(void* workspace, size_t* bytes, size_t need, moe_status* st) {
    if (need < kAlign) need = kAlign;  // never 0: a buffer sized from the query is not NULL
    if (!workspace) {
        *bytes = need;
        *st = MOE_OK;
        return true;
    }
    if ((uintptr_t)workspace & (kAlign - 1)) *st = MOE_ERR_INVALID_ARG;
    else if (*bytes < need) *st = MOE_ERR_WORKSPACE;
    else return false;
    return true;
}

}  // namespace moe
