// grouped.hpp -- what the kernels of the matrix products grouped by expert
// share: their arguments, the row lookups and the search of a tile's expert.
#pragma once

#include "common.hpp"
#include "launch.hpp"

namespace moe {

// moe_align's slot p = t*topk + j of sorted row i; anything outside
// [0, slots) marks a padding row.  p / topk by a multiplication: with
// magic = ceil(2^32 / topk) the product's upper half is exact for p*topk <
// 2^32, that is for the fewer than 2^28 slots the entry points accept.
// (topk == 1 has no 32-bit magic; its quotient is p.)
__device__ __forceinline__ uint32_t grouped_token(uint32_t p, uint32_t magic) {
    return __umulhi(p, magic) + (magic ? 0u : p);
}

// Row of a gathered / scattered / plain operand for sorted row i, -1 for
// padding.
__device__ __forceinline__ int grouped_row(const GroupedArgs& g, int i, uint32_t how) {
    if (!g.sorted) return i;
    const uint32_t p = (uint32_t)g.sorted[i];
    if (p >= g.slots) return -1;
    if (how == kRowToken) return (int)grouped_token(p, g.magic);
    return how == kRowSlot ? (int)p : i;
}

// Offsets are read clamped to [0, R], so that no list of offsets takes an
// access out of the R rows.
__device__ __forceinline__ int grouped_offset(const GroupedArgs& g, int e) {
    return min(max(g.offsets[e], 0), g.R);
}

// the same of a wave-uniform expert, by a scalar load (no kernel writes the
// offsets): it neither waits for nor counts with the vector loads and stores
// in flight
__device__ __forceinline__ int grouped_offset_scalar(const GroupedArgs& g, int e) {
    typedef const __attribute__((address_space(4))) int32_t* scalar_t;
    return min(max(((scalar_t)g.offsets)[e], 0), g.R);
}

// Which of the 64 rows of a block from its row `first` on are padding rows that
// the product writes: bit i for row first + i.  They are zeros whatever the
// weights hold (a row of zeros times an infinity would be NaN).  Scattered
// outputs drop them.  Called by all 64 lanes of a wave.
__device__ __forceinline__ uint64_t grouped_padding(const GroupedArgs& g, int row0, int rows, int first) {
    if (!g.sorted || g.how_out == kRowSlot) return 0;
    return __ballot((uint32_t)g.sorted[row0 + min(first + lane_id(), rows - 1)] >= g.slots);
}

// Rows products cut into g.splits ranges of the reduction leave an fp32 product
// [R, grouped_part_ld(width)] a range; rows stay 16-byte aligned.
__host__ __device__ inline int grouped_part_ld(int width) { return (width + 3) / 4 * 4; }
// range sp's steps [first, first + count) of `steps`
struct GroupedRange { int first, count; };
__host__ __device__ inline GroupedRange grouped_range(int steps, int splits, int sp) {
    const int per = (steps + splits - 1) / splits;
    const int first = sp * per < steps ? sp * per : steps;
    return {first, steps - first < per ? steps - first : per};
}

struct GroupedBlock {
    int e;       // expert, -1: no such block
    int row0;    // first sorted row of the block
    int rows;    // rows of it (<= the block size)
};

// The list that gives every expert ceil(rows / B) blocks, in expert order,
// spread over a wave: a lane holds four experts' offsets and block counts.
struct GroupedScan {
    int off[5], nb[4];
    int start;   // the lane's first block
    int total;   // blocks of all experts (wave-uniform)
};

// called by all 64 lanes of a wave
__device__ __forceinline__ GroupedScan grouped_scan(const GroupedArgs& g, int B) {
    const int lane = lane_id();
    GroupedScan s;
    int sum = 0;
#pragma unroll
    for (int j = 0; j < 5; ++j) s.off[j] = grouped_offset(g, min(4 * lane + j, g.E));
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int c = max(s.off[j + 1] - s.off[j], 0);
        s.nb[j] = (int)(((uint32_t)c + (uint32_t)B - 1) / (uint32_t)B);
        sum += s.nb[j];
    }
    // inclusive sum over the wave: within rows of 16 lanes, then the rows' ends on
    int incl = sum;
    incl += __builtin_amdgcn_update_dpp(0, incl, 0x111, 0xf, 0xf, false);  // row_shr:1
    incl += __builtin_amdgcn_update_dpp(0, incl, 0x112, 0xf, 0xf, false);  // row_shr:2
    incl += __builtin_amdgcn_update_dpp(0, incl, 0x114, 0xf, 0xf, false);  // row_shr:4
    incl += __builtin_amdgcn_update_dpp(0, incl, 0x118, 0xf, 0xf, false);  // row_shr:8
    incl += __builtin_amdgcn_update_dpp(0, incl, 0x142, 0xa, 0xf, false);  // row_bcast:15 to rows 1, 3
    incl += __builtin_amdgcn_update_dpp(0, incl, 0x143, 0xc, 0xf, false);  // row_bcast:31 to rows 2, 3
    // ascending offsets never reach the bound, which the launch grids cover
    s.total = min(__builtin_amdgcn_readlane(incl, kWave - 1), g.R / B + min(g.R, g.E));
    s.start = incl - sum;
    return s;
}

// block `blk` of the list (wave-uniform, as is the result)
__device__ __forceinline__ GroupedBlock grouped_find(const GroupedScan& s, int blk, int B) {
    int start = s.start, e = -1, row0 = 0, rows = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (blk >= start && blk < start + s.nb[j]) {
            e = 4 * lane_id() + j;
            row0 = s.off[j] + (blk - start) * B;
            rows = min(s.off[j + 1] - row0, B);
        }
        start += s.nb[j];
    }
    GroupedBlock r = {-1, 0, 0};
    const uint64_t hit = __ballot(e >= 0);
    if (hit) {
        const int l = __builtin_ctzll(hit);
        r.e = __builtin_amdgcn_readlane(e, l);
        r.row0 = __builtin_amdgcn_readlane(row0, l);
        r.rows = __builtin_amdgcn_readlane(rows, l);
    }
    return r;
}

}  // namespace moe
