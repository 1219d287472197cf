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
// the first n < 8 of 8 values, as 4, 2 and 1 of them
__device__ __forceinline__ void st_part(uint16_t* p, int n, uint4 w) {
    typedef uint32_t uint_any_t __attribute__((aligned(2)));
    if (n & 4) {
        *reinterpret_cast<u16x4_any_t*>(p) = __builtin_bit_cast(u16x4_t, uint2{w.x, w.y});
        p += 4;
        w.x = w.z;
        w.y = w.w;
    }
    if (n & 2) {
        *reinterpret_cast<uint_any_t*>(p) = w.x;
        p += 2;
        w.x = w.y;
    }
    if (n & 1) *p = (uint16_t)w.x;
}
template <bool ANY, bool ONCE = false>
__device__ __forceinline__ void st_bf16(uint16_t* p, int n, const float (&f)[V]) {
    u16x8_t v;
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = f32_to_bf16_bits(f[i]);
    if constexpr (!ANY && ONCE) __builtin_nontemporal_store(v, reinterpret_cast<u16x8_t*>(p));
    else if constexpr (!ANY) *reinterpret_cast<u16x8_t*>(p) = v;
    else if (n >= V) *reinterpret_cast<u16x8_any_t*>(p) = v;
    else st_part(p, n, __builtin_bit_cast(uint4, v));
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

// The bits of n of 8 columns of a row, zeros past them.  wide: the row has 8
// columns or more, and its last ones are loaded as its last 8 and moved into place.
template <bool ANY, bool ONCE = false>
__device__ __forceinline__ u16x8_t ld_bf16_bits(const uint16_t* p, int n, bool wide) {
    u16x8_t v = {0, 0, 0, 0, 0, 0, 0, 0};
    if constexpr (!ANY) {
        if (n <= 0) return v;
        if constexpr (ONCE) return __builtin_nontemporal_load(reinterpret_cast<const u16x8_t*>(p));
        else return *reinterpret_cast<const u16x8_t*>(p);
    } else if (n >= V) {
        v = *reinterpret_cast<const u16x8_any_t*>(p);
    } else if (wide && n > 0) {
        const int by = V - n;  // elements to drop in front
        uint4 w = __builtin_bit_cast(uint4, (u16x8_t)*reinterpret_cast<const u16x8_any_t*>(p - by));
        if (by & 4) w = uint4{w.z, w.w, 0, 0};
        if (by & 2) w = uint4{w.y, w.z, w.w, 0};
        if (by & 1)
            w = uint4{w.x >> 16 | w.y << 16, w.y >> 16 | w.z << 16, w.z >> 16 | w.w << 16, w.w >> 16};
        v = __builtin_bit_cast(u16x8_t, w);
    } else {
#pragma unroll
        for (int i = 0; i < V - 1; ++i)
            if (i < n) v[i] = p[i];
    }
    return v;
}
template <bool ANY, bool ONCE = false>
__device__ __forceinline__ void ld_bf16(const uint16_t* p, int n, bool wide, float (&f)[V]) {
    const u16x8_t v = ld_bf16_bits<ANY, ONCE>(p, n, wide);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = bf16_bits_to_f32(v[i]);
}

}  // namespace moe
