// tiles.hpp -- what the kernels with LDS-staged MFMA tiles share: bounds-checked
// buffer descriptors, the LDS row swizzle, and waits.
#pragma once

#include "common.hpp"

namespace moe {

typedef __amdgpu_buffer_rsrc_t prsrc_t;

__device__ __forceinline__ prsrc_t pmake_rsrc(const void* base, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
}
// an offset that no descriptor covers (all are below 2 GiB): reads give zeros,
// stores are dropped
constexpr uint32_t kNowhere = 0x80000000u;
__device__ __forceinline__ f32x16_t mfma32_bf16(bf16x8_t a, bf16x8_t b, f32x16_t c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// LDS rows: each operand row of a K-step is its BK elements (64 or 128
// bytes) without padding, its 16-byte chunks permuted by an XOR of the row
// index (swz, keyed by the chunks per row) so
// that the 16 consecutive rows an MFMA operand read touches in one LDS cycle
// land in distinct banks.  The DMA writes 1 KB per wave instruction in lane
// order, so lane l of an instruction covering rows r0.. stores physical
// chunk (l % CPR) of row r0 + l / CPR and therefore fetches logical chunk
// (l % CPR) ^ swz(row) from global memory.
template <int CPR>
__device__ __forceinline__ int swz(int r) {
    static_assert(CPR == 4 || CPR == 8, "64- or 128-byte LDS rows");
    if constexpr (CPR == 4) return ((r >> 1) & 3) ^ ((r >> 3) & 1);
    else return (r & 7) ^ ((r >> 3) & 1);
}

// s_waitcnt vmcnt(N) leaving the LDS/export counters unconstrained.
template <int N>
__device__ __forceinline__ void wait_vmcnt() {
    static_assert(N >= 0 && N < 64, "vmcnt range");
    __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | (7 << 4) | (15 << 8));
}

// The wave's LDS accesses issued so far are complete (lgkmcnt(0)), and the
// compiler moves no memory access across this point.  A wave's LDS
// instructions execute in order, so after it the wave's lanes read what its
// other lanes wrote before it.
__device__ __forceinline__ void lds_wave_fence() {
    __asm__ volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
}

// v, computed where it is used: an epilogue address derived from it is not
// hoisted to the kernel's start, where it would hold a register through the
// main loop (the ping-pong loops use all 256)
__device__ __forceinline__ int late_uniform(int v) {
    __asm__ volatile("" : "+s"(v));
    return v;
}

// the lane's index, computed where it is used: per-lane epilogue addresses
// are not hoisted to the kernel's start, where they would hold registers
// through the main loop
__device__ __forceinline__ int late_lane() {
    int v;
    __asm__ volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(v));
    return v;
}

}  // namespace moe
