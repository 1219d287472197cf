// small_tiles.hpp -- 64 x 64 pieces of an operand in LDS, for the kernels that load
// their tiles through registers: chunks of 8 elements from rows of any width and
// the fragments of 16x16x32 MFMAs.
//
// LDS layouts of 64 rows (or of 64 columns; 128 are two such parts), both 64
// rows of 128 bytes.  Rows along the output (operands that are contiguous in
// the reduction): 16-byte chunks permuted by the row as in the full tiles,
// fragments read directly.  Rows along the reduction: fragments come through
// the transposing read (lane i of 16 gets column i of four rows, that is 32
// bytes of each), 32-byte pieces permuted so that the two times four rows of a
// half-wave's read fall in different banks.
#pragma once

#include "common.hpp"
#include "tiles.hpp"

namespace moe {

constexpr int kSim = 64;                       // tile and step
constexpr int kSimBytes = kSim * kSim * 2;     // one operand's step

// What a kernel knows of the widths: multiples of 8, at least 8, or nothing.
enum class Widths { kWhole, kLong, kAny };

// What chunks outside an operand are loaded from, as one vector of 16 bytes: a
// branch a chunk costs more (us, with branches / so: 406 rows over 7 experts of
// 1001 x 330, dx 14.7/11.5; 4096 rows over 8 of 4097 x 2049, looked up, dw in bf16
// 177/164; but 16 rows over 8 of 14337 x 4095, forward 176/186)
alignas(16) static __device__ const uint16_t kZeros[8] = {0, 0, 0, 0, 0, 0, 0, 0};

// Columns c..c+7 of a row of `width`, zeros past its end and for no row.  A
// row's last chunk is loaded as the row's last 8 values, so that nothing past
// the row is read, and moved into place by settle_chunk when it is stored (a
// move here would wait for the load).
template <Widths W>
__device__ __forceinline__ u16x8_t load_chunk(const uint16_t* row, int c, int width) {
    const bool in = row && c < width;
    if constexpr (W == Widths::kWhole) {
        typedef const __attribute__((address_space(1))) u16x8_t* global_t;
        return *(global_t)(uintptr_t)(in ? row + c : kZeros);
    } else {
        if (W == Widths::kAny && width < 8) {
            u16x8_t v = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
            for (int i = 0; i < 7; ++i)
                if (row && c + i < width) v[i] = row[c + i];
            return v;
        }
        typedef const __attribute__((address_space(1))) u16x8_any_t* global_t;
        return *(global_t)(uintptr_t)(in ? row + min(c, width - 8) : kZeros);
    }
}
__device__ __forceinline__ u16x8_t settle_chunk(u16x8_t v, int c, int width) {
    const int by = width < 8 ? 0 : max(c - (width - 8), 0);  // elements to drop in front (0..7)
    uint4 w = __builtin_bit_cast(uint4, v);
    if (by & 4) w = uint4{w.z, w.w, 0, 0};
    if (by & 2) w = uint4{w.y, w.z, w.w, 0};
    if (by & 1) w = uint4{w.x >> 16 | w.y << 16, w.y >> 16 | w.z << 16, w.z >> 16 | w.w << 16, w.w >> 16};
    return __builtin_bit_cast(u16x8_t, w);
}

// chunk c (of 8) of row r, by layout
template <bool COL>
__device__ __forceinline__ int sim_at(int r, int c) {
    if constexpr (COL) {
        const int x = ((r >> 1) & 1) | (((r >> 3) & 1) << 1);
        return r * 128 + ((((c >> 1) ^ x) << 1 | (c & 1)) << 4);
    } else {
        return r * 128 + ((c ^ swz<8>(r)) << 4);
    }
}
// the fragment of 16 output rows / columns from `first`, k-slice ks
template <bool COL>
__device__ __forceinline__ bf16x8_t sim_frag(const char* buf, int first, int ks, int lane) {
    if constexpr (COL) {
        typedef short s16x4_t __attribute__((ext_vector_type(4)));
        typedef __attribute__((address_space(3))) s16x4_t* lp_t;
        const int q = lane >> 4, j = lane & 15;
        const int x = ((j >> 3) & 1) | ((q & 1) << 1);
        const char* p = buf + (ks * 32 + 8 * q + (j >> 2)) * 128 + (((first >> 4) ^ x) << 5) + (j & 3) * 8;
        const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp_t)p);
        const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp_t)(p + 4 * 128));
        return bf16x8_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    } else {
        return *reinterpret_cast<const bf16x8_t*>(buf + sim_at<false>(first + (lane & 15), ks * 4 + (lane >> 4)));
    }
}

}  // namespace moe
