// rows.hpp -- loads and stores of the kernels that go over rows elementwise:
// 8 columns a thread, 16 bytes of bf16.
#pragma once

#include "common.hpp"

namespace moe {

constexpr int V = 8;  // columns a thread takes at a time

// ANY: rows that are no multiple of 8 long.  Their columns are loaded and stored
// at any element address (vectors of 16 bytes all the same), the n < 8 columns
// that end a row one by one; the values of columns past the end are zero.
//
// ONCE: nothing of the line is used again on this XCD soon, and it need not
// stay in the L2 (rows of whole vectors only: others share lines).
typedef f32x4_t f32x4_any_t __attribute__((aligned(4)));

template <bool ANY, bool ONCE = false>
__device__ __forceinline__ void ld_bf16(const uint16_t* p, int n, float (&f)[V]) {
    u16x8_t v = {0, 0, 0, 0, 0, 0, 0, 0};
    if constexpr (!ANY && ONCE) v = __builtin_nontemporal_load(reinterpret_cast<const u16x8_t*>(p));
    else if constexpr (!ANY) v = *reinterpret_cast<const u16x8_t*>(p);
    else if (n >= V) v = *reinterpret_cast<const u16x8_any_t*>(p);
    else {
#pragma unroll
        for (int i = 0; i < V - 1; ++i)
            if (i < n) v[i] = p[i];
    }
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = bf16_bits_to_f32(v[i]);
}
template <bool ANY, bool ONCE = false>
__device__ __forceinline__ void st_bf16(uint16_t* p, int n, const float (&f)[V]) {
    u16x8_t v;
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = f32_to_bf16_bits(f[i]);
    if constexpr (!ANY && ONCE) __builtin_nontemporal_store(v, reinterpret_cast<u16x8_t*>(p));
    else if constexpr (!ANY) *reinterpret_cast<u16x8_t*>(p) = v;
    else if (n >= V) *reinterpret_cast<u16x8_any_t*>(p) = v;
    else {
#pragma unroll
        for (int i = 0; i < V - 1; ++i)
            if (i < n) p[i] = v[i];
    }
}
template <bool ANY>
__device__ __forceinline__ void ld_f32(const float* p, int n, float (&f)[V]) {
    if (ANY && n < V) {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = i < n ? p[i] : 0.0f;
        return;
    }
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        f32x4_t v;
        if constexpr (ANY) v = *reinterpret_cast<const f32x4_any_t*>(p + i);
        else v = *reinterpret_cast<const f32x4_t*>(p + i);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[i + j] = v[j];
    }
}
template <bool ANY, bool ONCE = false>
__device__ __forceinline__ void st_f32(float* p, int n, const float (&f)[V]) {
    if (ANY && n < V) {
#pragma unroll
        for (int i = 0; i < V - 1; ++i)
            if (i < n) p[i] = f[i];
        return;
    }
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        const f32x4_t v = {f[i], f[i + 1], f[i + 2], f[i + 3]};
        if constexpr (ANY) *reinterpret_cast<f32x4_any_t*>(p + i) = v;
        else if constexpr (ONCE) __builtin_nontemporal_store(v, reinterpret_cast<f32x4_t*>(p + i));
        else *reinterpret_cast<f32x4_t*>(p + i) = v;
    }
}

// the bits of n of 8 columns of a row, zeros past them
template <bool ANY, bool ONCE = false>
__device__ __forceinline__ u16x8_t ld_bf16_bits(const uint16_t* p, int n) {
    u16x8_t v = {0, 0, 0, 0, 0, 0, 0, 0};
    if constexpr (!ANY) {
        if (n <= 0) return v;
        if constexpr (ONCE) return __builtin_nontemporal_load(reinterpret_cast<const u16x8_t*>(p));
        else return *reinterpret_cast<const u16x8_t*>(p);
    } else if (n >= V) {
        v = *reinterpret_cast<const u16x8_any_t*>(p);
    } else {
#pragma unroll
        for (int i = 0; i < V - 1; ++i)
            if (i < n) v[i] = p[i];
    }
    return v;
}
}  // namespace moe
