// grouped_tiles.hip -- the grouped products on full 256 x 256 tiles, for
// widths that are multiples of 8 (rows of whole 16-byte chunks).
//
// A workgroup of 8 waves computes 256 output columns (operand A, on the MFMA
// row dimension) x 256 rows (operand B) with 32x32x16 bf16 MFMAs, 64 reduction
// elements a step.  The waves form two groups of four, a phase apart: while one
// group reads the next step's fragments from LDS, copies and waits, the other
// keeps the matrix cores busy (the schedule of the layer's own full tiles, see
// PingPongCore in gemm_prefill.hip, with operands of either orientation):
//
//   fwd  A = W[e] rows n (K contiguous)      B = x rows       (K contiguous)
//   dx   A = W[e] columns k (N strided)      B = dy rows      (N contiguous)
//   dw   A = x columns k (rows strided)      B = dy columns n (rows strided)
//
// "Row" operands hold the reduction contiguously: a step is 256 rows of 128
// bytes, fragments are 16-byte LDS reads.  "Column" operands hold it strided: a
// step is 64 rows of 512 bytes and fragments come through the transposing LDS
// read, which hands lane i of 16 the column i of four rows; the 64-byte pieces
// of a row are permuted by the row index, so that the four rows of such a read
// lie in different banks.  Nothing is transposed in memory.
//
// Every copy goes global -> LDS through a bounds-checked descriptor: rows past
// the end of an operand, reduction tails and padding rows are offsets out of
// its range, which leave zeros in LDS, so ragged sizes cost no branches in the
// main loop.  Column tails of "column" operands may copy a neighbouring row's
// values; they only reach outputs that are not stored.
#include "grouped.hpp"
#include "tiles.hpp"

#include <type_traits>

namespace moe {

namespace {

constexpr int kTile = 256, kStep = 64;
constexpr int kSlotBytes = kTile * kStep * 2;         // one operand's step
constexpr int kASlots = 3, kBSlots = 2;
constexpr int kLds = (kASlots + kBSlots) * kSlotBytes;
constexpr int kInstr = kSlotBytes / 1024 / 4;         // copies of a wave per step
// output tiles of one A column group that consecutive tiles share (see tile order below)
constexpr int kGroup = 4;
constexpr int kCusPerXcd = 32;

// Copies of an operand's step.  A wave copies one operand, 1 KB an instruction
// and kInstr of them a step; off[q] is the lane's source offset of copy q,
// held once for either kind of operand.
typedef uint32_t Offsets[kInstr];

// "Row" operand: 256 rows of 64 reduction elements from a descriptor that
// covers the tile's rows (or, for gathered rows, the whole operand).
struct RowCopy {
    prsrc_t r;
    uint32_t red_bytes;
    int first = 0;        // step of the reduction that counts as step 0

    // row of the tile that the lane's copy q fills, and its chunk of the
    // row: physical chunk lane % 8; the swizzle is the same for every q
    __device__ static __forceinline__ int row(int q, int gw, int lane) {
        return (q * 4 + gw) * 8 + lane / 8;
    }
    __device__ static __forceinline__ uint32_t chunk(int gw, int lane) {
        return (uint32_t)(((lane & 7) ^ swz<8>(gw * 8 + lane / 8)) << 4);
    }
    __device__ __forceinline__ void copy(const Offsets& off, char* slot, int step, int gw) const {
        typedef __attribute__((address_space(3))) void* lds_ptr_t;
        const uint32_t kb = (uint32_t)(first + step) * (kStep * 2);
        // the last step of a reduction that is no multiple of 64
        const bool cut = kb + kStep * 2 > red_bytes && kb + chunk(gw, late_lane()) >= red_bytes;
#pragma unroll
        for (int q = 0; q < kInstr; ++q)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)(slot + (q * 4 + gw) * 1024), 16,
                                                     cut ? kNowhere : off[q] + kb, 0, 0, 0);
    }
};

// "Column" operand: 64 rows of 256 columns, 16 consecutive rows a wave, two an
// instruction.  Row 16*gw + 2*q + lane/32 has its 64-byte pieces permuted by
// its low three bits, 2*(q%4) + lane/32.
struct ColCopy {
    const char* base;     // the tile's first column in row 0
    uint32_t ld;          // bytes a row
    uint32_t col0;        // bytes before the tile's first column in a row
    int red;              // rows
    int first = 0;        // step of the reduction that counts as step 0

    // the lane's chunk of its row at copy q
    __device__ static __forceinline__ uint32_t chunk(int q, int lane) {
        return ((uint32_t)((((lane & 31) >> 2) ^ (lane >> 5)) << 6) | (uint32_t)((lane & 3) << 4)) ^
               (uint32_t)((q & 3) << 7);
    }
    // offsets of rows in order, from a step's first row
    __device__ static __forceinline__ void in_order(Offsets& off, uint32_t ld, int gw, int lane) {
#pragma unroll
        for (int q = 0; q < kInstr; ++q)
            off[q] = (uint32_t)(gw * 16 + 2 * q + (lane >> 5)) * ld + chunk(q, lane);
    }
    __device__ static __forceinline__ void issue(const prsrc_t r, const Offsets& off, char* slot,
                                                 int gw) {
        typedef __attribute__((address_space(3))) void* lds_ptr_t;
#pragma unroll
        for (int q = 0; q < kInstr; ++q)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)(slot + (gw * 8 + q) * 1024), 16,
                                                     off[q], 0, 0, 0);
    }
    // the descriptor starts at the step's first row, so that offsets stay
    // small however many rows there are
    __device__ __forceinline__ void copy(const Offsets& off, char* slot, int step, int gw) const {
        const int row0 = (first + step) * kStep;
        const uint32_t rows = (uint32_t)min(red - row0, kStep);
        issue(pmake_rsrc(base + (size_t)row0 * ld, rows * ld - col0), off, slot, gw);
    }
};

// LDS byte offsets, within a slot, of a lane's fragments
template <bool COL, int NF>
struct Frag {
    // row: offset of k-slice ks of the first fragment, the others 32 rows on;
    // column: offset of fragment f, rows 0..3 of its 8 (4..7: ^256, +2048), k-slices 8 KB apart
    int off[COL ? NF : kStep / 16];

    __device__ __forceinline__ void init(int first_row, int lane) {
        const int li = lane & 31, half = lane >> 5;
        if constexpr (COL) {
            const int x = (lane & 15) >> 2;
#pragma unroll
            for (int f = 0; f < NF; ++f)
                off[f] = (8 * half + x) * 512 + (((first_row / 32 + f) ^ x) << 6) +
                         32 * ((lane >> 4) & 1) + 8 * (lane & 3);
        } else {
            const int r = first_row + li;
#pragma unroll
            for (int ks = 0; ks < kStep / 16; ++ks)
                off[ks] = r * 128 + (((2 * ks + half) ^ swz<8>(r)) << 4);
        }
    }
    __device__ __forceinline__ bf16x8_t read(const char* slot, int f, int ks) const {
        if constexpr (COL) {
            typedef short s16x4_t __attribute__((ext_vector_type(4)));
            typedef __attribute__((address_space(3))) s16x4_t* lp_t;
            const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lp_t)(slot + off[f] + ks * 16 * 512));
            const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                (lp_t)(slot + (off[f] ^ 256) + 2048 + ks * 16 * 512));
            return bf16x8_t{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        } else {
            return *reinterpret_cast<const bf16x8_t*>(slot + off[ks] + f * 32 * 128);
        }
    }
};

// A memory phase: the step's fragments from slots `a` and `b`, and `copy` into
// slot `to`.  The three slots are different ones, and saying so matters: the
// transposing read is known to the compiler as an access that copies in flight
// might still change, and it would wait for all of them before each phase.
// That a step's copies have landed is this file's waits and barriers.
template <bool ACOL, bool BCOL, typename Copy>
__device__ __forceinline__ bool memory_phase(bool compute, const char* __restrict__ a,
                                             const char* __restrict__ b, char* __restrict__ to,
                                             const Frag<ACOL, 4>& ra, const Frag<BCOL, 2>& rb,
                                             bf16x8_t (&fa)[4][4], bf16x8_t (&fb)[4][2],
                                             const Copy& copy) {
    if (compute) {
#pragma unroll
        for (int ks = 0; ks < 4; ++ks) {
#pragma unroll
            for (int f = 0; f < 4; ++f) fa[ks][f] = ra.read(a, f, ks);
#pragma unroll
            for (int f = 0; f < 2; ++f) fb[ks][f] = rb.read(b, f, ks);
        }
    }
    return copy(to);
}

// The main loop (phases and slot reuse as PingPongCore): operand B is copied by
// waves 0-3 one step ahead into two slots, operand A by waves 4-7 two steps
// ahead into three.
template <bool ACOL, bool BCOL, typename CopyA, typename CopyB>
struct PingPong {
    f32x16_t acc[4][2];

    __device__ __forceinline__ void finish(int wave) {
        if (wave < 4) __builtin_amdgcn_s_barrier();
    }

    template <bool COMPUTE>
    __device__ __forceinline__ void run(char* lds, const CopyA& ca, const CopyB& cb, const Offsets& off,
                                        int steps, int wave, int arow0, int brow0) {
        const int lane = lane_id();
        const bool second = wave >= 4;  // wave-uniform
        const int gw = wave & 3;
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[a][b][v] = 0.0f;
        auto slot_a = [&](int s) { return lds + s * kSlotBytes; };
        auto slot_b = [&](int s) { return lds + (kASlots + s) * kSlotBytes; };
        auto barrier = [&]() {
            __builtin_amdgcn_sched_barrier(0);
            __builtin_amdgcn_s_barrier();
            __builtin_amdgcn_sched_barrier(0);
        };
        Frag<ACOL, 4> ra;
        Frag<BCOL, 2> rb;
        ra.init(arow0, lane);
        rb.init(brow0, lane);
        bf16x8_t fa[4][4], fb[4][2];

        barrier();
        if (!second) {
            if (steps > 0) cb.copy(off, slot_b(0), 0, gw);
            wait_vmcnt<0>();
        } else {
            if (steps > 0) ca.copy(off, slot_a(0), 0, gw);
            if (steps > 1) {
                ca.copy(off, slot_a(1), 1, gw);
                wait_vmcnt<kInstr>();
            } else {
                wait_vmcnt<0>();
            }
        }
        barrier();
        if (second) barrier();
        int asl = 0, bsl = 0;
        for (int s = 0; s < steps; ++s) {
            // ---- memory phase
            const bool copied = memory_phase(
                COMPUTE, slot_a(asl), slot_b(bsl), second ? slot_a(asl == 0 ? 2 : asl - 1) : slot_b(bsl ^ 1),
                ra, rb, fa, fb, [&](char* to) {
                    const int n = s + (second ? 2 : 1);
                    if (n >= steps) return false;
                    if (second) ca.copy(off, to, n, gw);
                    else cb.copy(off, to, n, gw);
                    return true;
                });
            if (second) {
                if (copied) wait_vmcnt<kInstr>();
                else wait_vmcnt<0>();
            }
            __builtin_amdgcn_s_waitcnt(0xC07F);
            barrier();
            // ---- compute phase
            if constexpr (COMPUTE) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                    for (int a = 0; a < 4; ++a)
#pragma unroll
                        for (int b = 0; b < 2; ++b)
                            acc[a][b] = mfma32_bf16(fa[ks][a], fb[ks][b], acc[a][b]);
            }
            if (!second) wait_vmcnt<0>();
            barrier();
            asl = asl + 1 == kASlots ? 0 : asl + 1;
            bsl ^= 1;
        }
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b) pin(acc[a][b]);
    }
};

// ---- epilogue -----------------------------------------------------------------
// A wave's 64 B rows x 128 A columns go out through its own LDS area (the
// copies' slots are idle by then), so that a store instruction writes four
// rows' whole 256-byte segments instead of 8 or 16 bytes of each of 32 rows.
// `dst` gives the lane's B row's place in the output (in elements), negative
// for none.  Results do not stay in the L2, where the next tiles' operands are
// (8192 rows over 8 experts of 4096 x 512: 48.3 us, 50.9 in ordinary stores).
constexpr int kStRow = 256 + 16, kStArea = 64 * kStRow + 64 * 8;
static_assert(4 * kStArea <= kLds, "the staging fits the slots");

template <bool F32>
__device__ __forceinline__ void store_tile(char* st, const f32x16_t (&acc)[4][2], long dst, int c0,
                                           int cols, void* out) {
    const int lane = late_lane();
    const int li = lane & 31, half = lane >> 5, rr = lane >> 4, c = lane & 15;
    long* place = reinterpret_cast<long*>(st + 64 * kStRow);
    lds_wave_fence();
    place[lane] = dst;
    if constexpr (F32) {
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int a = 0; a < 2; ++a)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const f32x16_t& v = acc[2 * pass + a][b];
                        *reinterpret_cast<f32x4_t*>(st + (b * 32 + li) * kStRow +
                                                    (a * 32 + 8 * g + 4 * half) * 4) =
                            f32x4_t{v[4 * g], v[4 * g + 1], v[4 * g + 2], v[4 * g + 3]};
                    }
            lds_wave_fence();
            const int col = c0 + pass * 64 + c * 4;
#pragma unroll 4
            for (int i = 0; i < 16; ++i) {
                const int row = 4 * i + rr;
                const f32x4_t v = *reinterpret_cast<const f32x4_t*>(st + row * kStRow + c * 16);
                const long d = place[row];
                if (d >= 0 && col < cols) *reinterpret_cast<f32x4_t*>((float*)out + d + col) = v;
            }
            lds_wave_fence();
        }
    } else {
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const f32x16_t& v = acc[a][b];
                    uint2 p = {pack_bf16x2(v[4 * g], v[4 * g + 1]),
                               pack_bf16x2(v[4 * g + 2], v[4 * g + 3])};
                    *reinterpret_cast<uint2*>(st + (b * 32 + li) * kStRow +
                                              (a * 32 + 8 * g + 4 * half) * 2) = p;
                }
        lds_wave_fence();
        const int col = c0 + c * 8;
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {
            const int row = 4 * i + rr;
            const i32x4_t v = *reinterpret_cast<const i32x4_t*>(st + row * kStRow + c * 16);
            const long d = place[row];
            if (d >= 0 && col < cols)
                __builtin_nontemporal_store(v, reinterpret_cast<i32x4_t*>((uint16_t*)out + d + col));
        }
        lds_wave_fence();
    }
}

// ---- rows products ----------------------------------------------------------------
// Tile order: the hardware deals workgroup g to XCD g % 8.  Each XCD gets a
// contiguous range of tiles, numbered with kGroup column tiles fastest, then
// the experts' row blocks, so that the workgroups resident on an XCD share the
// weights and rows they copy in its L2.  The number of row blocks is known on
// the device only: the grid covers the most there can be.
//
// Few tiles: PARTS cuts the reduction into g.splits ranges, each of which
// stores its fp32 product of the tile; rows_join adds them up.
template <bool DX, bool LOOK, bool PARTS>
__global__ __launch_bounds__(512, 2) void grouped_rows_kernel(GroupedArgs g) {
    __shared__ __attribute__((aligned(1024))) char lds[kLds];
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int gw = wave & 3;
    const int cols = DX ? g.K : g.N, red = DX ? g.N : g.K;
    const int a_tiles = (cols + kTile - 1) / kTile;
    const GroupedScan scan = grouped_scan(g, kTile);
    const int tiles = a_tiles * scan.total, total = PARTS ? tiles * g.splits : tiles;
    const int per_xcd = (total + 7) / 8;
    const int local = (int)blockIdx.x / 8;
    int t = ((int)blockIdx.x % 8) * per_xcd + local;
    if (local >= per_xcd || t >= total) return;
    const int sp = PARTS ? t / tiles : 0;
    if constexpr (PARTS) t %= tiles;
    const int span = kGroup * scan.total;
    const int grp = t / span, in = t % span;
    const int gsize = min(kGroup, a_tiles - grp * kGroup);
    const int a0 = (grp * kGroup + in % gsize) * kTile;
    const GroupedBlock blk = grouped_find(scan, in / gsize, kTile);

    const uint16_t* w = g.w + (size_t)blk.e * g.N * g.K;
    const uint16_t* src = DX ? g.dy : g.x;
    const uint32_t how = DX ? g.how_dy : g.how_x;
    const uint32_t ld_b = (uint32_t)red * 2;
    typedef typename std::conditional<DX, ColCopy, RowCopy>::type CopyA;
    CopyA ca;
    RowCopy cb;
    Offsets off;
    if constexpr (DX) {
        ca.base = (const char*)(w + a0);
        ca.ld = (uint32_t)g.K * 2;
        ca.col0 = (uint32_t)a0 * 2;
        ca.red = red;
    } else {
        ca.r = pmake_rsrc(w + (size_t)a0 * g.K, (uint32_t)min(cols - a0, kTile) * ld_b);
        ca.red_bytes = ld_b;
    }
    const bool by_token = LOOK && how == kRowToken;
    cb.r = pmake_rsrc(by_token ? src : src + (size_t)blk.row0 * red,
                      (uint32_t)(by_token ? g.T : blk.rows) * ld_b);
    cb.red_bytes = ld_b;
    if (DX && wave >= 4) {
        if constexpr (DX) ColCopy::in_order(off, ca.ld, gw, lane);
    } else {
        const uint32_t chunk = RowCopy::chunk(gw, lane);
        uint32_t p[kInstr];
        if constexpr (LOOK) {
#pragma unroll
            for (int q = 0; q < kInstr; ++q)  // in flight together
                p[q] = (uint32_t)g.sorted[blk.row0 + min(RowCopy::row(q, gw, lane), blk.rows - 1)];
        }
#pragma unroll
        for (int q = 0; q < kInstr; ++q) {
            uint32_t j = (uint32_t)RowCopy::row(q, gw, lane);
            bool ok = true;  // past the tile's rows the descriptor ends
            if (LOOK && wave < 4) {
                ok = (j < (uint32_t)blk.rows) & (p[q] < g.slots);
                if (by_token) j = grouped_token(p[q], g.magic);
            }
            off[q] = ok ? j * ld_b + chunk : kNowhere;
        }
    }
    // wave tile: 128 columns x 64 rows, 2 x 2 waves in each half of the rows
    const int arow0 = (gw & 1) * 128, brow0 = (wave >> 2) * 128 + (gw >> 1) * 64;
    const bool used = brow0 < blk.rows;
    const uint64_t padding = LOOK ? grouped_padding(g, blk.row0, blk.rows, brow0) : 0;
    int steps = (red + kStep - 1) / kStep;
    if constexpr (PARTS) {
        const GroupedRange range = grouped_range(steps, g.splits, sp);
        ca.first = cb.first = range.first;
        steps = range.count;
    }
    PingPong<DX, false, CopyA, RowCopy> core;
    if (used) core.template run<true>(lds, ca, cb, off, steps, wave, arow0, brow0);
    else core.template run<false>(lds, ca, cb, off, steps, wave, arow0, brow0);
    if (used) {
        if (__builtin_expect(padding != 0, 0)) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
                if (padding >> (32 * b + (late_lane() & 31)) & 1) {
#pragma unroll
                    for (int a = 0; a < 4; ++a) core.acc[a][b] = f32x16_t{};
                }
        }
        const int j = brow0 + late_lane();
        long row = -1;
        if (j < blk.rows)
            row = !PARTS && g.how_out == kRowSlot ? grouped_row(g, blk.row0 + j, kRowSlot) : blk.row0 + j;
        if (PARTS && row >= 0) row += (long)sp * g.R;
        store_tile<PARTS>(lds + gw * kStArea, core.acc, row < 0 ? -1 : row * cols, a0 + arow0, cols,
                          g.out);
    }
    core.finish(wave);
}

// ---- weight gradient -----------------------------------------------------------------
// An expert's reduction is its rows, often few steps long, so a tile's start
// (the first copies' latency) and end (256 x 256 values to store) would cost as
// much as its products.  A workgroup therefore stays for many tiles and its
// copies run on from one tile into the next: the ring of slots knows steps
// only, and while a tile's results are stored the next tile's first two steps
// are in flight.  Per tile each group's phases are (memory, compute) for every
// step and one more that stores, the second group a phase behind as above:
//
//   first     M0 C0 .. Ms-1 Cs-1 E    M0'  C0'
//   second       M0 .. Cs-2 Ms-1 Cs-1 E    M0'
//
// Both groups stage their results through the slot of operand A's last step,
// the only one that no copy in flight uses, 8 KB a wave: the first group's E
// runs while the second computes from registers, the second's while the first
// reads other slots.  Waits count in the order of issue, so a copy issued after
// a tile's stores would land only when those are done: the first group issues
// the one of its next memory phase before its stores (its slot is free once
// both groups have read the tile's last step), and the second group, whose
// copies lead by two steps, waits for all but the stores and the last copy.
//
// Looked-up rows: a step's slots come by scalar loads a phase before they are
// used, their offsets are computed between the MFMAs of the compute phase.
//
// 8192 rows over 8 experts of 28672 x 4096: 1780-1810 us (1070 TFLOP/s with 1.9
// GB of results; a library product of 8192^3 in this orientation 1037).  What
// costs is the ends of tiles of 16 steps: storing one adds 3-4 us to its 31
// (32768 rows, 14336 x 4096: 3.05 ms, 1260 TFLOP/s).  Looked-up rows take 7 %
// more (1930-1960 us): their scalar work is issued between the MFMAs, and with
// half as much of it again they took 10 %.  The looked-up case in one run by its
// output: bf16 2.00 ms, fp32 2.16 and added to fp32 2.74 (plain rows 2.50), whose
// stores wait for what was there eight times a tile, with five registers spilled
// where rows are looked up.
//
// Tile order: each XCD takes an eighth of every expert's tiles (experts have
// different numbers of rows; an expert to an XCD would leave most of them
// idle), the eighths turned from expert to expert so that few tiles spread too
// -- not by one each, as a workgroup's tiles lie a multiple of eight experts
// apart when there are few (488 rows over 245 experts of 576 x 192: 59.0 us by
// one, 29.7 as here); within it kGroup column tiles fastest, then the n tiles.
// Few output tiles over many rows: an expert's rows are cut into g.splits ranges
// of whole steps, each a "part" e * splits + s with its own fp32 product in the
// workspace; dw_join adds them up in order.  (1024 x 1024 over 8192 rows of one
// expert: 213 us in one range, 42 us in 16.)
struct DwTile {
    int e, a0, b0, row0, rows;   // e: the part
};
template <bool PARTS>
__device__ __forceinline__ void dw_rows(const GroupedArgs& g, int part, int& row0, int& rows) {
    const int e = PARTS ? part / g.splits : part, s = PARTS ? part % g.splits : 0;
    row0 = grouped_offset_scalar(g, e);
    rows = max(grouped_offset_scalar(g, e + 1) - row0, 0);
    if constexpr (PARTS) {
        const int steps = (rows + kStep - 1) / kStep;
        const int len = (steps + g.splits - 1) / g.splits * kStep;
        const int from = min(s * len, rows);
        row0 += from;
        rows = min(rows - from, len);
    }
}
template <bool PARTS>
struct DwWalk {
    int a_tiles, b_tiles, tiles, per_xcd, xcd, stride, end;

    __device__ __forceinline__ DwWalk(const GroupedArgs& g) {
        a_tiles = (g.K + kTile - 1) / kTile;
        b_tiles = (g.N + kTile - 1) / kTile;
        tiles = a_tiles * b_tiles;
        per_xcd = (tiles + 7) / 8;
        xcd = (int)blockIdx.x % 8;
        stride = (int)gridDim.x / 8;
        end = g.E * (PARTS ? g.splits : 1) * per_xcd;
    }
    // the first tile at or after position `at` of this workgroup's list (with
    // rows, if `rows_only`); at is end when there is none
    __device__ __forceinline__ DwTile find(const GroupedArgs& g, int& at, bool rows_only) const {
        DwTile t = {0, 0, 0, 0, 0};
        for (; at < end; at += stride) {
            t.e = at / per_xcd;
            const int i = ((xcd + t.e + t.e / 8 + t.e / 32) % 8) * per_xcd + at % per_xcd;
            if (i >= tiles) continue;
            dw_rows<PARTS>(g, t.e, t.row0, t.rows);
            if (rows_only && t.rows == 0) continue;
            const int span = kGroup * b_tiles, grp = i / span, in = i % span;
            const int gsize = min(kGroup, a_tiles - grp * kGroup);
            t.a0 = (grp * kGroup + in % gsize) * kTile;
            t.b0 = in / gsize * kTile;
            return t;
        }
        at = end;
        return t;
    }
};
// The steps of a workgroup's tiles, one after the other.
struct DwSteps {
    int at, step;
    DwTile t;

    template <typename Walk>
    __device__ __forceinline__ bool more(const Walk& w) const { return at < w.end; }
    template <typename Walk>
    __device__ __forceinline__ void next(const GroupedArgs& g, const Walk& w) {
        if (++step * kStep >= t.rows) {
            at += w.stride;
            t = w.find(g, at, true);
            step = 0;
        }
    }
};

constexpr int kDwStores = 16;  // stores of a wave's results, at least
constexpr int kNonTemporal = 2;  // of a buffer instruction's cache policy

// Rows n0.. (of at most 64) and columns k0.. (of 128) of dW[e] from a wave's
// accumulators, through 8 KB of LDS: 32 rows of 256 bytes at a time, chunks
// permuted by the row.  Every store is issued whatever the tile's size (what
// lies outside is an offset out of range), so that their number is known.  They
// leave the L2 to the operands (2048 rows over 8 experts of 14336 x 4096: 316 us,
// 365 in ordinary stores).
typedef __attribute__((address_space(3))) char* lds_char_t;

// ds_write_b64 / b128 without the wait for copies in flight that the compiler
// puts before a store to LDS; the caller fences
__device__ __forceinline__ void stage(uint32_t at, uint2 v) {
    __asm__ volatile("ds_write_b64 %0, %1" ::"v"(at), "v"(v) : "memory");
}
__device__ __forceinline__ void stage(uint32_t at, f32x4_t v) {
    __asm__ volatile("ds_write_b128 %0, %1" ::"v"(at), "v"(v) : "memory");
}
// v, used from here on as if it were another value: addresses made from it are
// computed again instead of being held in registers that the main loop needs
__device__ __forceinline__ uint32_t fresh(uint32_t v) {
    __asm__ volatile("" : "+v"(v));
    return v;
}

enum class DwOut { kBf16, kF32, kF32Add, kParts };  // kParts: fp32, of the rows' ranges
template <DwOut OUT>
__device__ __forceinline__ void store_dw(char* st, const f32x16_t (&acc)[4][2],
                                         const GroupedArgs& g, int e, int n0, int k0) {
    const int lane = late_lane();
    const int li = lane & 31, half = lane >> 5, rr = lane >> 4, c = lane & 15;
    constexpr int size = OUT == DwOut::kBf16 ? 2 : 4, per = 16 / size;
    const uint32_t ld = (uint32_t)(g.K * size);
    char* base = (char*)g.out + (((size_t)e * g.N + n0) * g.K + k0) * size;
    const prsrc_t r = pmake_rsrc(base, (uint32_t)min(64, g.N - n0) * ld - (uint32_t)(k0 * size));
    const uint32_t at = (uint32_t)rr * ld + (uint32_t)(c * 16);
    // (st is 8 KB aligned: the permutations are XORs of bits 4..7)
    const uint32_t base_st = (uint32_t)(uintptr_t)(lds_char_t)st;
    const uint32_t put = base_st + (uint32_t)(li * 256) +
                         (OUT == DwOut::kBf16 ? ((li & 15) << 4) + 8 * half : ((li & 15) ^ half) << 4);
    const uint32_t get = base_st + (uint32_t)(rr * 256 + ((c ^ rr) << 4));
    auto flush = [&](int row0, int col0) {
        lds_wave_fence();
        __builtin_amdgcn_sched_barrier(0);
        const uint32_t from = fresh(get), to = fresh(at);
        const bool in = k0 + col0 + c * per < g.K;
#pragma unroll
        for (int i0 = 0; i0 < 8; i0 += 4) {
            i32x4_t v[4], was[4];
            uint32_t o[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {  // row 4*(i0 + i) + rr
                v[i] = *(const __attribute__((address_space(3))) i32x4_t*)(lds_char_t)(
                    (uintptr_t)((from ^ (uint32_t)(i << 6)) + (uint32_t)((i0 + i) * 1024)));
                o[i] = in ? to + (uint32_t)(row0 + 4 * (i0 + i)) * ld + (uint32_t)(col0 * size)
                          : kNowhere;
                if constexpr (OUT == DwOut::kF32Add)
                    was[i] = __builtin_amdgcn_raw_buffer_load_b128(r, o[i], 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (OUT == DwOut::kF32Add) {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[i][j] = __float_as_int(__int_as_float(was[i][j]) + __int_as_float(v[i][j]));
                }
                __builtin_amdgcn_raw_buffer_store_b128(v[i], r, o[i], 0, kNonTemporal);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        lds_wave_fence();
        __builtin_amdgcn_sched_barrier(0);
    };
#pragma unroll
    for (int b = 0; b < 2; ++b) {
        if constexpr (OUT != DwOut::kBf16) {
#pragma unroll
            for (int pass = 0; pass < 2; ++pass) {
                const uint32_t w = fresh(put);
#pragma unroll
                for (int a = 0; a < 2; ++a)
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const f32x16_t& v = acc[2 * pass + a][b];
                        stage(w ^ (uint32_t)((a * 8 + 2 * q) << 4),
                              f32x4_t{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]});
                        __builtin_amdgcn_sched_barrier(0);
                    }
                flush(b * 32, pass * 64);
            }
        } else {
            const uint32_t w = fresh(put);
#pragma unroll
            for (int a = 0; a < 4; ++a)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const f32x16_t& v = acc[a][b];
                    stage(w ^ (uint32_t)((a * 4 + q) << 4),
                          uint2{pack_bf16x2(v[4 * q], v[4 * q + 1]),
                                pack_bf16x2(v[4 * q + 2], v[4 * q + 3])});
                    __builtin_amdgcn_sched_barrier(0);
                }
            flush(b * 32, 0);
        }
    }
}

// the same rows and columns as zeros, without LDS; `zeros`: accumulators of no steps
__device__ __forceinline__ void store_dw_zeros(const f32x16_t& zeros, const GroupedArgs& g, int e,
                                               int n0, int k0) {
    const int lane = late_lane(), size = g.out_f32 ? 4 : 2, lg = g.out_f32 ? 5 : 4;  // 2^lg chunks a row
    const uint32_t ld = (uint32_t)(g.K * size);
    char* base = (char*)g.out + (((size_t)e * g.N + n0) * g.K + k0) * size;
    const prsrc_t r = pmake_rsrc(base, (uint32_t)min(64, g.N - n0) * ld - (uint32_t)(k0 * size));
    const uint32_t c = (uint32_t)(lane & ((1 << lg) - 1)) * 16;
    // rows past the last are out of range
    uint32_t at = c < (uint32_t)(min(128, g.K - k0) * size) ? (uint32_t)(lane >> lg) * ld + c : kNowhere;
    const i32x4_t z = __builtin_bit_cast(i32x4_t, f32x4_t{zeros[0], zeros[1], zeros[2], zeros[3]});
#pragma unroll 1
    for (int i = 0; i < 1 << lg; ++i, at += (uint32_t)(kWave >> lg) * ld)
        __builtin_amdgcn_raw_buffer_store_b128(z, r, at, 0, 0);
}

template <bool LOOK, DwOut OUT>
__global__ __launch_bounds__(512, 2) void grouped_dw_kernel(GroupedArgs g) {
    __shared__ __attribute__((aligned(1024))) char lds[kLds];
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int gw = wave & 3;
    const bool second = wave >= 4;
    const DwWalk<OUT == DwOut::kParts> walk(g);
    auto slot_a = [&](int s) { return lds + s * kSlotBytes; };
    auto slot_b = [&](int s) { return lds + (kASlots + s) * kSlotBytes; };
    auto barrier = [&]() {
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_sched_barrier(0);
    };
    // a wave copies one operand: waves 4-7 x (A) two steps ahead, waves 0-3 dy
    // (B) one step ahead
    const uint16_t* src = second ? g.x : g.dy;
    const int width = second ? g.K : g.N;
    const uint32_t ld = (uint32_t)width * 2;
    const bool token = LOOK && (second ? g.how_x : g.how_dy) == kRowToken;
    Offsets off;
    if constexpr (!LOOK) ColCopy::in_order(off, ld, gw, lane);
    // slots of the rows that this wave copies next (wave-uniform scalar loads)
    typedef const __attribute__((address_space(4))) int32_t* scalar_t;
    int ids[LOOK ? 16 : 1];
    DwSteps lead = {(int)blockIdx.x / 8, 0, {}};  // the step copied next
    lead.t = walk.find(g, lead.at, true);
    auto look = [&]() {
        if constexpr (LOOK) {
            if (!lead.more(walk)) return;
            const int first = lead.step * kStep + gw * 16;
            const scalar_t p = (scalar_t)(g.sorted + lead.t.row0);
            if (first + 16 <= lead.t.rows) {
#pragma unroll
                for (int i = 0; i < 16; ++i) ids[i] = p[first + i];
            } else {  // past the last row: no slot
#pragma unroll
                for (int i = 0; i < 16; ++i)
                    ids[i] = p[min(first + i, lead.t.rows - 1)] | (first + i < lead.t.rows ? 0 : -1);
            }
        }
    };
    // a row's place: the slot's token (a quotient, see grouped_token; topk == 1
    // as 2p * 2^31) or its position in the step.  Scalar work as far as it
    // goes, and little of it: it has to fit between the MFMAs
    const uint32_t quot = !token ? 0 : g.magic ? g.magic : 1u << 31, shift = token && !g.magic;
    const uint32_t in_step = token ? 0 : (uint32_t)(gw * 16 + (lane >> 5)) * ld, two_rows = token ? 0 : 2 * ld;
    const uint32_t chunk0 = ColCopy::chunk(0, lane);
    // offsets of copy q from its two rows' slots
    auto place = [&](int q) {
        if constexpr (LOOK) {
            uint32_t o[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t p = (uint32_t)ids[2 * q + h];
                const uint32_t at = __umulhi(p << shift, quot) * ld;
                o[h] = p < g.slots ? at : kNowhere;
            }
            // (from their first forms each time: held for every q they would cost
            // registers that the loop does not have)
            off[q] = (lane >> 5 ? o[1] : o[0]) + (fresh(in_step) + (uint32_t)q * two_rows) +
                     (fresh(chunk0) ^ (uint32_t)((q & 3) << 7));
        }
    };
    auto place_all = [&]() {
#pragma unroll
        for (int q = 0; q < kInstr; ++q) place(q);
    };
    // copies the lead step into `slot` and moves on; false: none left
    auto copy_next = [&](char* slot) {
        if (!lead.more(walk)) return false;
        const uint32_t first = (uint32_t)(second ? lead.t.a0 : lead.t.b0);
        const int row0 = lead.step * kStep;
        const uint32_t rows = (uint32_t)min(lead.t.rows - row0, kStep);
        const uint32_t all = g.T > 0 ? (uint32_t)g.T : 0;
        const uint16_t* p = src + first + (token ? 0 : (size_t)(lead.t.row0 + row0) * width);
        const uint32_t bytes = (token ? all : rows) * ld;
        ColCopy::issue(pmake_rsrc(p, bytes ? bytes - first * 2 : 0), off, slot, gw);
        lead.next(g, walk);
        look();
        return true;
    };

    const int arow0 = (gw & 1) * 128, brow0 = (wave >> 2) * 128 + (gw >> 1) * 64;
    Frag<true, 4> ra;
    Frag<true, 2> rb;
    ra.init(arow0, lane);
    rb.init(brow0, lane);
    bf16x8_t fa[4][4], fb[4][2];
    f32x16_t acc[4][2];
    look();
    place_all();
    copy_next(second ? slot_a(0) : slot_b(0));
    place_all();
    if (second) {
        copy_next(slot_a(1));
        place_all();
    }
    wait_vmcnt<0>();
    barrier();
    if (second) barrier();
    int asl = 0, bsl = 0;
    bool stored = false;  // the phase before issued kDwStores stores or more
    bool early = false;   // the next memory phase's copy is issued already
    for (int at = (int)blockIdx.x / 8;; at += walk.stride) {
        const DwTile t = walk.find(g, at, OUT == DwOut::kF32Add);
        if (at >= walk.end) break;
        const bool used = t.b0 + brow0 < g.N && t.a0 + arow0 < g.K;
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b)
#pragma unroll
                for (int v = 0; v < 16; ++v) acc[a][b][v] = 0.0f;
        for (int left = t.rows; left > 0; left -= kStep) {
            // ---- memory phase
            const bool copied = memory_phase(
                used, slot_a(asl), slot_b(bsl),
                second ? slot_a(asl == 0 ? 2 : asl - 1) : slot_b(bsl ^ 1), ra, rb, fa, fb,
                [&](char* to) { return early || copy_next(to); });
            if (second) {
                // the next step has landed: only this copy, and the stores
                // issued after the one before it, may be left
                if (!copied) wait_vmcnt<0>();
                else if (stored) wait_vmcnt<kInstr + kDwStores>();
                else wait_vmcnt<kInstr>();
            }
            __builtin_amdgcn_s_waitcnt(0xC07F);
            barrier();
            // ---- compute phase
            if (used) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks)
#pragma unroll
                    for (int a = 0; a < 4; ++a) {
#pragma unroll
                        for (int b = 0; b < 2; ++b)
                            acc[a][b] = mfma32_bf16(fa[ks][a], fb[ks][b], acc[a][b]);
                        if constexpr (LOOK) {
                            if (a & 1) {
                                place(ks * 2 + a / 2);
                                __builtin_amdgcn_sched_barrier(0);
                            }
                        }
                    }
            } else {
                place_all();
            }
            if (!second) {
                // the next step has landed; its copy is older than the stores
                if (early && stored) wait_vmcnt<kDwStores>();
                else wait_vmcnt<0>();
            }
            early = stored = false;
            barrier();
            asl = asl + 1 == kASlots ? 0 : asl + 1;
            bsl ^= 1;
        }
#pragma unroll
        for (int a = 0; a < 4; ++a)
#pragma unroll
            for (int b = 0; b < 2; ++b) pin(acc[a][b]);
        // ---- the tile's results
        if (!second && !early) {
            copy_next(slot_b(bsl ^ 1));
            early = true;
        }
        if (used) {
            if (OUT != DwOut::kF32Add && t.rows == 0) {  // (kF32Add walks tiles with rows only)
                store_dw_zeros(acc[0][0], g, t.e, t.b0 + brow0, t.a0 + arow0);
            } else {
                store_dw<OUT>(slot_a(asl == 0 ? 2 : asl - 1) + gw * (kSlotBytes / 4), acc, g, t.e,
                              t.b0 + brow0, t.a0 + arow0);
                stored = true;
            }
        }
        barrier();
    }
    if (!second) barrier();  // for the second group's phase behind
}

}  // namespace

// Rows whose slots have to be looked up to read them: gathered rows, and
// padding rows that count as zeros (a scattered output drops them instead).
static bool rows_look(const GroupedArgs& g, uint32_t how) {
    return g.sorted && !(how == kRowSorted && g.how_out == kRowSlot);
}

int grouped_tiles_rows_workgroups(const GroupedArgs& g, bool dx) {
    const int a_tiles = ((dx ? g.K : g.N) + kTile - 1) / kTile;
    const long most = (long)a_tiles * (g.R / kTile + (g.R < g.E ? g.R : g.E));
    return (int)((most * g.splits + 7) / 8 * 8);
}

template <bool DX>
static void launch_rows_tiles(const GroupedArgs& g, hipStream_t s) {
    const int grid = grouped_tiles_rows_workgroups(g, DX);
    auto run = [&](auto look, auto parts) {
        grouped_rows_kernel<DX, decltype(look)::value, decltype(parts)::value><<<grid, 512, 0, s>>>(g);
    };
    const std::true_type yes;
    const std::false_type no;
    if (rows_look(g, DX ? g.how_dy : g.how_x)) g.splits > 1 ? run(yes, yes) : run(yes, no);
    else g.splits > 1 ? run(no, yes) : run(no, no);
}
void launch_grouped_tiles_fwd(const GroupedArgs& g, hipStream_t s) { launch_rows_tiles<false>(g, s); }
void launch_grouped_tiles_dx(const GroupedArgs& g, hipStream_t s) { launch_rows_tiles<true>(g, s); }

namespace {
// out = (out +) the parts' products, in order; a thread per four values
template <DwOut OUT>
__global__ __launch_bounds__(256) void dw_join_kernel(const float* __restrict__ parts, int splits,
                                                      size_t per_expert, size_t total, void* out) {
    const size_t at = ((size_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (at >= total) return;
    const size_t e = at / per_expert;
    const float* p = parts + e * (splits - 1) * per_expert + at;  // (e*splits)*per + at % per
    f32x4_t v = *reinterpret_cast<const f32x4_t*>(p);
    for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const f32x4_t*>(p + s * per_expert);
    if constexpr (OUT == DwOut::kBf16) {
        uint2 q = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        *reinterpret_cast<uint2*>((uint16_t*)out + at) = q;
    } else {
        f32x4_t* o = reinterpret_cast<f32x4_t*>((float*)out + at);
        *o = OUT == DwOut::kF32Add ? *o + v : v;
    }
}

long dw_tiles(const GroupedArgs& g) {
    return (long)((g.K + kTile - 1) / kTile) * ((g.N + kTile - 1) / kTile);
}
}  // namespace

// Ranges an expert's rows are cut into: until the tiles of the experts that can
// have rows fill the CUs, as long as a range keeps eight steps on average
// (2048 x 2 rows over 8 experts of 1024 x 256: 22.6 us whole, 27.8 us in two
// ranges of four steps).
int grouped_tiles_dw_splits(const GroupedArgs& g) {
    const long tiles = dw_tiles(g) * (g.R < g.E ? g.R : g.E);
    int splits = 1;
    while (splits < 16 && tiles * splits * 2 <= 8 * kCusPerXcd &&
           (long)g.R / (g.R < g.E ? g.R : g.E) / (splits * 2) >= 8 * kStep)
        splits *= 2;
    return splits;
}

int grouped_tiles_dw_workgroups(const GroupedArgs& g) {
    const long per_xcd = (dw_tiles(g) + 7) / 8 * g.E * g.splits;
    return 8 * (int)(per_xcd < kCusPerXcd ? per_xcd : kCusPerXcd);
}

void launch_grouped_tiles_dw(const GroupedArgs& call, void* workspace, hipStream_t s) {
    GroupedArgs g = call;
    if (g.splits > 1) {
        g.out = workspace;
        g.out_f32 = 1;
        g.accumulate = 0;
    }
    const int grid = grouped_tiles_dw_workgroups(g);
    auto run = [&](auto look, auto out) {
        grouped_dw_kernel<decltype(look)::value, decltype(out)::value><<<grid, 512, 0, s>>>(g);
    };
    auto with_out = [&](auto look) {
        if (g.splits > 1) run(look, std::integral_constant<DwOut, DwOut::kParts>{});
        else if (g.accumulate) run(look, std::integral_constant<DwOut, DwOut::kF32Add>{});
        else if (g.out_f32) run(look, std::integral_constant<DwOut, DwOut::kF32>{});
        else run(look, std::integral_constant<DwOut, DwOut::kBf16>{});
    };
    if (g.sorted) with_out(std::true_type{});
    else with_out(std::false_type{});
    if (g.splits > 1) {
        const size_t per = (size_t)g.N * g.K, total = per * g.E;
        const int blocks = (int)((total / 4 + 255) / 256);
        const float* parts = (const float*)workspace;
        if (call.accumulate)
            dw_join_kernel<DwOut::kF32Add><<<blocks, 256, 0, s>>>(parts, g.splits, per, total, call.out);
        else if (call.out_f32)
            dw_join_kernel<DwOut::kF32><<<blocks, 256, 0, s>>>(parts, g.splits, per, total, call.out);
        else
            dw_join_kernel<DwOut::kBf16><<<blocks, 256, 0, s>>>(parts, g.splits, per, total, call.out);
    }
}

}  // namespace moe
