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

// Where a tile's operand comes from.
struct Source {
    const char* base;   // row: first row of the tile; column: row 0 of the reduction, tile's column
    uint32_t bytes;     // row: covered from base; column, token rows: likewise
    uint32_t ld;        // bytes per row
    int red;            // reduction elements
    int col0;           // column: byte offset of the tile's first column within a row
};

template <bool LOOK>
struct RowCopy {
    prsrc_t r;
    uint32_t ld, red_bytes, lane_off, chunk;
    uint32_t off[LOOK ? kInstr : 1];

    // rows: row of lane's copy q in the operand (LOOK), -1 padding; else the tile's rows in order
    __device__ __forceinline__ void init(const Source& s, int gw, int lane) {
        r = pmake_rsrc(s.base, s.bytes);
        ld = s.ld;
        red_bytes = (uint32_t)s.red * 2;
        // row (q*4 + gw)*8 + lane/8: its swizzle is the same for every q
        chunk = (uint32_t)(((lane & 7) ^ swz<8>(gw * 8 + lane / 8)) << 4);
        lane_off = (uint32_t)(gw * 8 + lane / 8) * ld + chunk;
    }
    __device__ static __forceinline__ int row(int q, int gw, int lane) {
        return (q * 4 + gw) * 8 + lane / 8;
    }
    __device__ __forceinline__ void copy(char* slot, int step, int gw) const {
        typedef __attribute__((address_space(3))) void* lds_ptr_t;
        const uint32_t kb = (uint32_t)step * (kStep * 2);
        const bool out = kb + chunk >= red_bytes;  // false for every lane before the last step
#pragma unroll
        for (int q = 0; q < kInstr; ++q) {
            uint32_t v = LOOK ? off[q] : lane_off + (uint32_t)(q * 32) * ld;
            v = out ? kNowhere : v + kb;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)(slot + (q * 4 + gw) * 1024), 16,
                                                     v, 0, 0, 0);
        }
    }
};

template <bool LOOK>
struct ColCopy {
    // LOOK: the expert's slots, through the scalar loads of the constant address
    // space (no kernel writes them; vector loads would count with the copies)
    typedef const __attribute__((address_space(4))) int32_t* ids_t;
    const char* base;
    ids_t ids;
    uint32_t ld, bytes, lane_off, chunk, slots, magic;
    int red, col0, half;
    bool token;           // LOOK: rows by token (fixed base) or by position
    int next[LOOK ? 2 * kInstr : 1];

    __device__ __forceinline__ void init(const Source& s, int gw, int lane) {
        base = s.base;
        bytes = s.bytes;
        ld = s.ld;
        red = s.red;
        col0 = s.col0;
        half = lane >> 5;
        // row 2*(q*4 + gw) + lane/32 of the step; its low three bits are the same for every q
        const int x = (2 * gw + half) & 7;
        chunk = (uint32_t)(((((lane & 31) >> 2) ^ x) * 4 + (lane & 3)) << 4);
        lane_off = (uint32_t)(2 * gw + half) * ld + chunk;
    }
    // the slots of the rows this wave copies at `step` (wave-uniform loads)
    __device__ __forceinline__ void look(int step, int gw) {
        if constexpr (LOOK) {
            const int last = red - 1;
#pragma unroll
            for (int q = 0; q < kInstr; ++q)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int i = step * kStep + 2 * (q * 4 + gw) + h;
                    next[2 * q + h] = last < 0 ? -1 : ids[min(i, last)];
                }
        }
    }
    __device__ __forceinline__ void copy(char* slot, int step, int gw) const {
        typedef __attribute__((address_space(3))) void* lds_ptr_t;
        const int row0 = step * kStep;
        const bool fixed = LOOK && token;
        // the descriptor starts at the step's first row, so that offsets stay
        // small however many rows the expert has
        const uint32_t rows = (uint32_t)min(red - row0, kStep);
        const prsrc_t r = pmake_rsrc(base + (fixed ? 0 : (size_t)row0 * ld),
                                     fixed ? bytes : rows * ld - (uint32_t)col0);
#pragma unroll
        for (int q = 0; q < kInstr; ++q) {
            uint32_t v;
            if constexpr (LOOK) {
                const int i = 2 * (q * 4 + gw) + half;
                const uint32_t p = (uint32_t)(half ? next[2 * q + 1] : next[2 * q]);
                const uint32_t row = token ? grouped_token(p, magic) : (uint32_t)i;
                v = p < slots && row0 + i < red ? row * ld + chunk : kNowhere;
            } else {
                v = lane_off + (uint32_t)(q * 8) * ld;
            }
            __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr_t)(slot + (q * 4 + gw) * 1024), 16,
                                                     v, 0, 0, 0);
        }
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
    __device__ __forceinline__ void run(char* lds, CopyA& ca, CopyB& cb, int steps, int wave,
                                        int arow0, int brow0) {
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
            if constexpr (BCOL) cb.look(0, gw);
            if (steps > 0) cb.copy(slot_b(0), 0, gw);
            if constexpr (BCOL) cb.look(1, gw);
            wait_vmcnt<0>();
        } else {
            if constexpr (ACOL) ca.look(0, gw);
            if (steps > 0) ca.copy(slot_a(0), 0, gw);
            if constexpr (ACOL) ca.look(1, gw);
            if (steps > 1) {
                ca.copy(slot_a(1), 1, gw);
                if constexpr (ACOL) ca.look(2, gw);
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
                    cb.copy(slot_b(bsl ^ 1), s + 1, gw);
                    if constexpr (BCOL) cb.look(s + 2, gw);
                }
            } else {
                if (s + 2 < steps) {
                    ca.copy(slot_a(asl == 0 ? 2 : asl - 1), s + 2, gw);
                    if constexpr (ACOL) ca.look(s + 3, gw);
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
    typedef typename std::conditional<DX, ColCopy<false>, RowCopy<false>>::type CopyA;
    typedef RowCopy<LOOK> CopyB;
    CopyA ca;
    CopyB cb;
    if constexpr (DX)
        ca.init(Source{(const char*)(w + a0), 0, (uint32_t)g.K * 2, red, a0 * 2}, gw, lane);
    else
        ca.init(Source{(const char*)(w + (size_t)a0 * g.K),
                       (uint32_t)min(cols - a0, kTile) * (uint32_t)(g.K * 2), (uint32_t)g.K * 2, red,
                       0}, gw, lane);
    const bool by_token = LOOK && how == kRowToken;
    cb.init(Source{(const char*)(by_token ? src : src + (size_t)blk.row0 * red),
                   (uint32_t)(by_token ? g.T : blk.rows) * ld_b, ld_b, red, 0}, gw, lane);
    if constexpr (LOOK) {
        uint32_t p[kInstr];
#pragma unroll
        for (int q = 0; q < kInstr; ++q)  // in flight together
            p[q] = (uint32_t)g.sorted[blk.row0 + min(CopyB::row(q, gw, lane), blk.rows - 1)];
#pragma unroll
        for (int q = 0; q < kInstr; ++q) {
            const int j = CopyB::row(q, gw, lane);
            const uint32_t row = by_token ? grouped_token(p[q], g.magic) : (uint32_t)j;
            cb.off[q] = j < blk.rows && p[q] < g.slots ? row * ld_b + cb.chunk : kNowhere;
        }
    }
    // wave tile: 128 columns x 64 rows, 2 x 2 waves in each half of the rows
    const int arow0 = (gw & 1) * 128, brow0 = (wave >> 2) * 128 + (gw >> 1) * 64;
    const bool used = brow0 < blk.rows;
    const int steps = (red + kStep - 1) / kStep;
    PingPong<DX, false, CopyA, CopyB> core;
    if (used) core.template run<true>(lds, ca, cb, steps, wave, arow0, brow0);
    else core.template run<false>(lds, ca, cb, steps, wave, arow0, brow0);
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

    typedef ColCopy<LOOK> Copy;
    auto source = [&](Copy& c, const uint16_t* p, int width, int first, uint32_t how) {
        const bool token = LOOK && how == kRowToken;
        const uint32_t ld = (uint32_t)width * 2;
        c.init(Source{(const char*)(p + (token ? 0 : (size_t)row0 * width) + first),
                      g.T > 0 ? (uint32_t)g.T * ld - (uint32_t)first * 2 : 0, ld, rows, first * 2},
               gw, lane);
        c.ids = (typename Copy::ids_t)(g.sorted + row0);
        c.slots = g.slots;
        c.magic = g.magic;
        c.token = token;
    };
    Copy ca, cb;
    source(ca, g.x, g.K, a0, g.how_x);
    source(cb, g.dy, g.N, b0, g.how_dy);
    const int arow0 = (gw & 1) * 128, brow0 = (wave >> 2) * 128 + (gw >> 1) * 64;
    const bool used = b0 + brow0 < g.N && a0 + arow0 < g.K;
    const int steps = (rows + kStep - 1) / kStep;
    PingPong<true, true, Copy, Copy> core;
    if (used) core.template run<true>(lds, ca, cb, steps, wave, arow0, brow0);
    else core.template run<false>(lds, ca, cb, steps, wave, arow0, brow0);
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
