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

constexpr uint32_t kNowhere = 0x80000000u;  // an offset no descriptor covers (all are below 2 GiB)
constexpr int kTile = 256, kStep = 64;
constexpr int kSlotBytes = kTile * kStep * 2;         // one operand's step
constexpr int kASlots = 3, kBSlots = 2;
constexpr int kLds = (kASlots + kBSlots) * kSlotBytes;
constexpr int kInstr = kSlotBytes / 1024 / 4;         // copies of a wave per step
// output tiles of one A column group that consecutive tiles share (see tile order below)
constexpr int kGroup = 4;

// Copies of an operand's step.  A wave copies one operand, 1 KB an instruction
// and kInstr of them a step; off[q] is the lane's source offset of copy q,
// held once for either kind of operand.
typedef uint32_t Offsets[kInstr];

// "Row" operand: 256 rows of 64 reduction elements from a descriptor that
// covers the tile's rows (or, for gathered rows, the whole operand).
struct RowCopy {
    static constexpr bool kLook = false;  // its lookups are done once, before the loop
    prsrc_t r;
    uint32_t red_bytes;

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
        const uint32_t kb = (uint32_t)step * (kStep * 2);
        // the last step of a reduction that is no multiple of 64
        const bool cut = kb + kStep * 2 > red_bytes && kb + chunk(gw, late_lane()) >= red_bytes;
#pragma unroll
        for (int q = 0; q < kInstr; ++q)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)(slot + (q * 4 + gw) * 1024), 16,
                                                     cut ? kNowhere : off[q] + kb, 0, 0, 0);
    }
};

// "Column" operand: 64 rows of 256 columns.  LOOK: a row is found by its slot
// -- the slot's token (`token`, rows anywhere in the operand), or its position,
// with padding rows as zeros; else rows in order.
template <bool LOOK>
struct ColCopy {
    static constexpr bool kLook = LOOK;
    const char* base;     // the tile's first column in the expert's first row (token: in row 0)
    const int32_t* ids;   // LOOK: the expert's slots
    uint32_t ld, bytes;   // bytes a row; token: bytes that base covers
    uint32_t col0;        // bytes before the tile's first column in a row
    uint32_t slots, magic;
    int red;              // rows
    bool token;

    // row 2*(q*4 + gw) + lane/32 of a step: its low three bits, the same for
    // every q, and the lane's chunk of it
    __device__ static __forceinline__ int low(int gw, int lane) { return 2 * gw + (lane >> 5); }
    __device__ static __forceinline__ uint32_t chunk(int gw, int lane) {
        return (uint32_t)(((((lane & 31) >> 2) ^ low(gw, lane)) * 4 + (lane & 3)) << 4);
    }
    __device__ __forceinline__ void in_order(Offsets& off, int gw, int lane) const {
#pragma unroll
        for (int q = 0; q < kInstr; ++q)
            off[q] = (uint32_t)(q * 8 + low(gw, lane)) * ld + chunk(gw, lane);
    }
    // Looking rows up takes three steps, so that none waits for memory: fetch
    // loads the slot of row `lane` of a step (one load a wave, a step before
    // its copy is placed), place turns it into the row's offset and hands each
    // lane those of the rows it copies, copy issues the copies.
    __device__ __forceinline__ int fetch(int step, int lane) const {
        return red > 0 ? ids[min(step * kStep + lane, red - 1)] : -1;
    }
    __device__ __forceinline__ void place(Offsets& off, int id, int step, int gw, int lane) const {
        const uint32_t p = (uint32_t)id;
        const uint32_t row = token ? grouped_token(p, magic) : (uint32_t)lane;
        const bool ok = (p < slots) & (step * kStep + lane < red);
        const uint32_t at = ok ? row * ld : kNowhere;
#pragma unroll
        for (int q = 0; q < kInstr; ++q)
            off[q] = (uint32_t)__builtin_amdgcn_ds_bpermute(4 * low(gw, lane) + 32 * q, (int)at) +
                     chunk(gw, lane);
    }
    __device__ __forceinline__ void copy(const Offsets& off, char* slot, int step, int gw) const {
        typedef __attribute__((address_space(3))) void* lds_ptr_t;
        const bool fixed = LOOK && token;
        const int row0 = step * kStep;
        // the descriptor starts at the step's first row, so that offsets stay
        // small however many rows there are
        const uint32_t rows = (uint32_t)min(red - row0, kStep);
        const prsrc_t r = pmake_rsrc(base + (fixed ? 0 : (size_t)row0 * ld),
                                     fixed ? bytes : rows * ld - col0);
#pragma unroll
        for (int q = 0; q < kInstr; ++q)
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)(slot + (q * 4 + gw) * 1024), 16,
                                                     off[q], 0, 0, 0);
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
    __device__ __forceinline__ void run(char* lds, const CopyA& ca, const CopyB& cb, Offsets& off,
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

        int id = -1;  // slot of the step after the next copy
        barrier();
        if (!second) {
            int id0 = -1;
            if constexpr (CopyB::kLook) {
                id0 = cb.fetch(0, lane);
                id = cb.fetch(1, lane);
                cb.place(off, id0, 0, gw, lane);
            }
            if (steps > 0) cb.copy(off, slot_b(0), 0, gw);
            if constexpr (CopyB::kLook) cb.place(off, id, 1, gw, lane);
            wait_vmcnt<0>();
        } else {
            int id0 = -1, id1 = -1;
            if constexpr (CopyA::kLook) {
                id0 = ca.fetch(0, lane);
                id1 = ca.fetch(1, lane);
                id = ca.fetch(2, lane);
                ca.place(off, id0, 0, gw, lane);
            }
            if (steps > 0) ca.copy(off, slot_a(0), 0, gw);
            if (steps > 1) {
                if constexpr (CopyA::kLook) ca.place(off, id1, 1, gw, lane);
                ca.copy(off, slot_a(1), 1, gw);
                if constexpr (CopyA::kLook) ca.place(off, id, 2, gw, lane);
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
            if constexpr (COMPUTE) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) {
#pragma unroll
                    for (int a = 0; a < 4; ++a) fa[ks][a] = ra.read(slot_a(asl), a, ks);
#pragma unroll
                    for (int b = 0; b < 2; ++b) fb[ks][b] = rb.read(slot_b(bsl), b, ks);
                }
            }
            if (!second) {
                if (s + 1 < steps) {
                    if constexpr (CopyB::kLook) id = cb.fetch(s + 2, lane);
                    cb.copy(off, slot_b(bsl ^ 1), s + 1, gw);
                }
            } else {
                if (s + 2 < steps) {
                    if constexpr (CopyA::kLook) id = ca.fetch(s + 3, lane);
                    ca.copy(off, slot_a(asl == 0 ? 2 : asl - 1), s + 2, gw);
                    wait_vmcnt<kInstr>();
                } else {
                    wait_vmcnt<0>();
                }
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
            if (!second) {
                if constexpr (CopyB::kLook) cb.place(off, id, s + 2, gw, lane);
                wait_vmcnt<0>();
            } else if constexpr (CopyA::kLook) {
                ca.place(off, id, s + 3, gw, lane);
            }
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
// for none.
constexpr int kStRow = 256 + 16, kStArea = 64 * kStRow + 64 * 8;
static_assert(4 * kStArea <= kLds, "the staging fits the slots");

__device__ __forceinline__ void store_tile(char* st, const f32x16_t (&acc)[4][2], long dst, int c0,
                                           int cols, void* out, int out_f32, int accumulate) {
    const int lane = late_lane();
    const int li = lane & 31, half = lane >> 5, rr = lane >> 4, c = lane & 15;
    long* place = reinterpret_cast<long*>(st + 64 * kStRow);
    lds_wave_fence();
    place[lane] = dst;
    if (out_f32) {
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
                f32x4_t v = *reinterpret_cast<const f32x4_t*>(st + row * kStRow + c * 16);
                const long d = place[row];
                if (d >= 0 && col < cols) {
                    f32x4_t* p = reinterpret_cast<f32x4_t*>((float*)out + d + col);
                    if (accumulate) v = *p + v;
                    *p = v;
                }
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
                *reinterpret_cast<i32x4_t*>((uint16_t*)out + d + col) = v;
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
template <bool DX, bool LOOK>
__global__ __launch_bounds__(512, 2) void grouped_rows_kernel(GroupedArgs g) {
    __shared__ __attribute__((aligned(1024))) char lds[kLds];
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int gw = wave & 3;
    const int cols = DX ? g.K : g.N, red = DX ? g.N : g.K;
    const int a_tiles = (cols + kTile - 1) / kTile;
    const GroupedScan scan = grouped_scan(g, kTile);
    const int total = a_tiles * scan.total;
    const int per_xcd = (total + 7) / 8;
    const int local = (int)blockIdx.x / 8;
    const int t = ((int)blockIdx.x % 8) * per_xcd + local;
    if (local >= per_xcd || t >= total) return;
    const int span = kGroup * scan.total;
    const int grp = t / span, in = t % span;
    const int gsize = min(kGroup, a_tiles - grp * kGroup);
    const int a0 = (grp * kGroup + in % gsize) * kTile;
    const GroupedBlock blk = grouped_find(scan, in / gsize, kTile);

    const uint16_t* w = g.w + (size_t)blk.e * g.N * g.K;
    const uint16_t* src = DX ? g.dy : g.x;
    const uint32_t how = DX ? g.how_dy : g.how_x;
    const uint32_t ld_b = (uint32_t)red * 2;
    typedef typename std::conditional<DX, ColCopy<false>, RowCopy>::type CopyA;
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
        if constexpr (DX) ca.in_order(off, gw, lane);
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
    const int steps = (red + kStep - 1) / kStep;
    PingPong<DX, false, CopyA, RowCopy> core;
    if (used) core.template run<true>(lds, ca, cb, off, steps, wave, arow0, brow0);
    else core.template run<false>(lds, ca, cb, off, steps, wave, arow0, brow0);
    if (used) {
        const int j = brow0 + late_lane();
        long row = -1;
        if (j < blk.rows)
            row = g.how_out == kRowSlot ? grouped_row(g, blk.row0 + j, kRowSlot) : blk.row0 + j;
        store_tile(lds + gw * kStArea, core.acc, row < 0 ? -1 : row * cols, a0 + arow0, cols, g.out,
                   0, 0);
    }
    core.finish(wave);
}

// ---- weight gradient -----------------------------------------------------------------
// Tile order: each XCD takes an eighth of every expert's tiles (experts have
// different numbers of rows; an expert to an XCD would leave most of them
// idle), the eighths turned by one from expert to expert so that few tiles
// spread too; within it kGroup column tiles fastest, then the n tiles.
template <bool LOOK>
__global__ __launch_bounds__(512, 2) void grouped_dw_kernel(GroupedArgs g) {
    __shared__ __attribute__((aligned(1024))) char lds[kLds];
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int gw = wave & 3;
    const int a_tiles = (g.K + kTile - 1) / kTile, b_tiles = (g.N + kTile - 1) / kTile;
    const int tiles = a_tiles * b_tiles, per_xcd = (tiles + 7) / 8;
    const int local = (int)blockIdx.x / 8;
    const int e = local / per_xcd;
    const int t = (((int)blockIdx.x + e) % 8) * per_xcd + local % per_xcd;
    if (e >= g.E || t >= tiles) return;
    const int span = kGroup * b_tiles;
    const int grp = t / span, in = t % span;
    const int gsize = min(kGroup, a_tiles - grp * kGroup);
    const int a0 = (grp * kGroup + in % gsize) * kTile, b0 = (in / gsize) * kTile;
    const int row0 = __builtin_amdgcn_readfirstlane(grouped_offset(g, e));
    const int rows = max(__builtin_amdgcn_readfirstlane(grouped_offset(g, e + 1)) - row0, 0);
    if (rows == 0 && g.accumulate) return;

    // a wave copies one operand: waves 4-7 x (A), waves 0-3 dy (B)
    const bool is_x = wave >= 4;
    const uint16_t* p = is_x ? g.x : g.dy;
    const int width = is_x ? g.K : g.N, first = is_x ? a0 : b0;
    const uint32_t ld = (uint32_t)width * 2;
    ColCopy<LOOK> copy;
    copy.token = LOOK && (is_x ? g.how_x : g.how_dy) == kRowToken;
    copy.base = (const char*)(p + (copy.token ? 0 : (size_t)row0 * width) + first);
    copy.ld = ld;
    copy.col0 = (uint32_t)first * 2;
    copy.bytes = g.T > 0 ? (uint32_t)g.T * ld - copy.col0 : 0;
    copy.red = rows;
    copy.ids = g.sorted + row0;
    copy.slots = g.slots;
    copy.magic = g.magic;
    Offsets off;
    if constexpr (!LOOK) copy.in_order(off, gw, lane);
    const int arow0 = (gw & 1) * 128, brow0 = (wave >> 2) * 128 + (gw >> 1) * 64;
    const bool used = b0 + brow0 < g.N && a0 + arow0 < g.K;
    const int steps = (rows + kStep - 1) / kStep;
    PingPong<true, true, ColCopy<LOOK>, ColCopy<LOOK>> core;
    if (used) core.template run<true>(lds, copy, copy, off, steps, wave, arow0, brow0);
    else core.template run<false>(lds, copy, copy, off, steps, wave, arow0, brow0);
    if (used) {
        const int n = b0 + brow0 + late_lane();
        store_tile(lds + gw * kStArea, core.acc, n < g.N ? ((long)e * g.N + n) * g.K : -1, a0 + arow0,
                   g.K, g.out, g.out_f32, g.accumulate);
    }
    core.finish(wave);
}

}  // namespace

// Rows whose slots have to be looked up to read them: gathered rows, and
// padding rows that count as zeros (a scattered output drops them instead).
static bool rows_look(const GroupedArgs& g, uint32_t how) {
    return g.sorted && !(how == kRowSorted && g.how_out == kRowSlot);
}

template <bool DX>
static void launch_rows_tiles(const GroupedArgs& g, hipStream_t s) {
    const int a_tiles = ((DX ? g.K : g.N) + kTile - 1) / kTile;
    const long most = (long)a_tiles * (g.R / kTile + (g.R < g.E ? g.R : g.E));
    const int grid = (int)((most + 7) / 8 * 8);
    if (rows_look(g, DX ? g.how_dy : g.how_x)) grouped_rows_kernel<DX, true><<<grid, 512, 0, s>>>(g);
    else grouped_rows_kernel<DX, false><<<grid, 512, 0, s>>>(g);
}
void launch_grouped_tiles_fwd(const GroupedArgs& g, hipStream_t s) { launch_rows_tiles<false>(g, s); }
void launch_grouped_tiles_dx(const GroupedArgs& g, hipStream_t s) { launch_rows_tiles<true>(g, s); }

void launch_grouped_tiles_dw(const GroupedArgs& g, hipStream_t s) {
    const long tiles = (long)((g.K + kTile - 1) / kTile) * ((g.N + kTile - 1) / kTile);
    const int grid = (int)((tiles + 7) / 8 * 8 * g.E);
    if (g.sorted) grouped_dw_kernel<true><<<grid, 512, 0, s>>>(g);
    else grouped_dw_kernel<false><<<grid, 512, 0, s>>>(g);
}

}  // namespace moe
