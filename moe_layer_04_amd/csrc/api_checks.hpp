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

struct Bytes {
    const void* p;
    long n;
};
// whether an output shares bytes with an input or with another output
template <int OUTS, int INS>
bool overlaps(const Bytes (&outs)[OUTS], const Bytes (&ins)[INS]) {
    for (int i = 0; i < OUTS; ++i) {
        if (!outs[i].p) continue;
        for (const Bytes& in : ins)
            if (in.p && overlap(outs[i].p, outs[i].n, in.p, in.n)) return true;
        for (int j = 0; j < i; ++j)
            if (outs[j].p && overlap(outs[i].p, outs[i].n, outs[j].p, outs[j].n)) return true;
    }
    return false;
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

// The size reported by a call that may not use its workspace: the minimum exactly
// if it does not, so that a caller may pass any buffer then.
inline size_t used_size(size_t need) {
    return need == 0 ? 0 : need < 2 * kAlign ? 2 * kAlign : round_up(need);
}

}  // namespace moe
