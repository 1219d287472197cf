// ckpt.hpp -- rows kept in 8 bits: blocks of 32 columns of a row share one byte X,
// a value is code * 2^(X-133) with a code of -127..127 (OCP MXINT8: an E8M0 scale
// and 8-bit integers of 6 fraction bits).
//
// X is the least byte with max |x| <= 127 * 2^(X-133), so the step is at most
// max |x| / 63.5 and a value is off by at most half of that.  A bf16 value has
// 8 significant bits, a code 7: every kept value is a bf16 number, and whoever
// reads it as one rounds nothing again.  X = 255: the block held an infinity or a
// NaN, and all its values are NaN.
#pragma once

#include "ckpt_sizes.hpp"
#include "rows.hpp"

namespace moe {

constexpr int kCkptLanes = kCkptBlock / V;  // a quad of lanes, 8 columns each, holds a block
constexpr uint32_t kCkptNan = 255;

typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));
typedef u32x2_t u32x2_any_t __attribute__((aligned(1)));

// X from the bits (without the sign) of a block's largest magnitude: 127 * 2^(X-133)
// is 2^(X-127) less one of its 128 steps, so X is the exponent field, and one
// more where all fraction bits are set.
__device__ __forceinline__ uint32_t ckpt_power(uint32_t top) {
    if (top >= 0x7f80u) return kCkptNan;
    return top < 128u ? 0u : min((top + 1u) >> 7, 254u);
}

// X of the block that this lane's quad holds (all four lanes active)
__device__ __forceinline__ uint32_t ckpt_quad_power(u16x8_t v) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < V; ++i) top = max(top, (uint32_t)v[i] & 0x7fffu);
    top = max(top, xchg_u32<0>(top));
    top = max(top, xchg_u32<1>(top));
    return ckpt_power(top);
}

// The codes of 8 values, the first in the lowest byte.  1.5 * 2^23 + q has q's
// low byte as its own, and the sum rounds to the nearest q, ties to even.  (Only
// X = 254 can round to 128.)
__device__ __forceinline__ u32x2_t ckpt_codes(u16x8_t v, uint32_t X) {
    uint32_t b[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const float q = __builtin_ldexpf(bf16_bits_to_f32(v[i]), 133 - (int)X);
        b[i] = __float_as_uint(__builtin_amdgcn_fmed3f(q, -127.0f, 127.0f) + 12582912.0f);
    }
    u32x2_t w;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const uint32_t lo = __builtin_amdgcn_perm(b[4 * h + 1], b[4 * h], 0x0c0c0400u);
        const uint32_t hi = __builtin_amdgcn_perm(b[4 * h + 3], b[4 * h + 2], 0x0c0c0400u);
        w[h] = X == kCkptNan ? 0u : __builtin_amdgcn_perm(hi, lo, 0x05040100u);
    }
    return w;
}

// 2^(X-133) in fp32 (subnormal below X = 7), NaN for X = 255
__device__ __forceinline__ float ckpt_step(uint32_t X) {
    const uint32_t bits = X >= 7u ? (X - 6u) << 23 : 1u << (16u + X);
    return __uint_as_float(X == kCkptNan ? 0x7fc00000u : bits);
}
// the 8 values of codes (exact: a product of a 7-bit integer and a power of two)
__device__ __forceinline__ void ckpt_values(u32x2_t w, uint32_t X, float (&f)[V]) {
    const float step = ckpt_step(X);
#pragma unroll
    for (int i = 0; i < V; ++i) f[i] = (float)(int8_t)(w[i / 4] >> (8 * (i % 4))) * step;
}

// n of 8 columns' codes (ANY, ONCE, wide: as in rows.hpp)
template <bool ANY, bool ONCE = false>
__device__ __forceinline__ u32x2_t ld_codes(const int8_t* p, int n, bool wide) {
    if constexpr (!ANY && ONCE) return __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(p));
    if constexpr (!ANY) return *reinterpret_cast<const u32x2_t*>(p);
    if (n >= V) return *reinterpret_cast<const u32x2_any_t*>(p);
    uint64_t b = 0;
    if (wide) {
        const int by = V - n;
        b = __builtin_bit_cast(uint64_t, (u32x2_t)*reinterpret_cast<const u32x2_any_t*>(p - by)) >> (8 * by);
    } else {
#pragma unroll
        for (int i = 0; i < V - 1; ++i)
            if (i < n) b |= (uint64_t)(uint8_t)p[i] << (8 * i);
    }
    return __builtin_bit_cast(u32x2_t, b);
}
template <bool ANY>
__device__ __forceinline__ void st_codes(int8_t* p, int n, u32x2_t w) {
    typedef uint32_t uint_any_t __attribute__((aligned(1)));
    typedef uint16_t ushort_any_t __attribute__((aligned(1)));
    if constexpr (!ANY) {
        *reinterpret_cast<u32x2_t*>(p) = w;
    } else if (n >= V) {
        *reinterpret_cast<u32x2_any_t*>(p) = w;
    } else {  // as 4, 2 and 1 of them
        uint32_t v = w[0];
        if (n & 4) {
            *reinterpret_cast<uint_any_t*>(p) = v;
            p += 4;
            v = w[1];
        }
        if (n & 2) {
            *reinterpret_cast<ushort_any_t*>(p) = (uint16_t)v;
            p += 2;
            v >>= 16;
        }
        if (n & 1) *p = (int8_t)v;
    }
}

}  // namespace moe
