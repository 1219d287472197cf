// grouped_gemm.hip -- matrix products grouped by expert over ragged row
// ranges: sorted row i of the range [offsets[e], offsets[e+1]) meets expert
// e's weights W[e] [N,K].
//
//   fwd  y[i,n]    = sum_k W[e][n,k] x[i,k]
//   dx   dx[i,k]   = sum_n W[e][n,k] dy[i,n]
//   dw   dW[e][n,k] = sum_{i of e} dy[i,n] x[i,k]
//
// Every product takes its two operands as "A" (the output's contiguous
// dimension, on the MFMA row dimension, so that a lane's accumulators are
// neighbours in memory) and "B" (the other one).  Row lookups (gather by
// token, scatter by slot) happen in the kernels; sums are fp32.
#include "grouped.hpp"

namespace moe {

namespace {

constexpr int kOpFwd = 0, kOpDx = 1, kOpDw = 2;

// ---------------------------------------------------------------------------
// Any widths: 64 x 64 outputs per workgroup of four waves, 32 reduction
// elements a step, element loads guarded one by one and staged through
// registers into LDS rows of 32 + 8 elements (the pad spreads the 16 rows of
// an operand read over the banks).  16x16x32 MFMA: lane l supplies row
// l % 16, reduction 8*(l/16)..+8; its accumulators are rows 4*(l/16)+v of
// column l % 16.
// ---------------------------------------------------------------------------
constexpr int kSimTile = 64, kSimStep = 32, kSimRow = kSimStep + 8;

template <int OP>
__global__ __launch_bounds__(256, 4) void grouped_any_kernel(GroupedArgs g) {
    __shared__ __attribute__((aligned(16))) uint16_t la[kSimTile * kSimRow];
    __shared__ __attribute__((aligned(16))) uint16_t lb[kSimTile * kSimRow];
    const int tid = (int)threadIdx.x, lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int a_dim = OP == kOpFwd ? g.N : g.K;
    const int a_tiles = (a_dim + kSimTile - 1) / kSimTile;
    const int a0 = ((int)blockIdx.x % a_tiles) * kSimTile;  // first output column
    const int bt = (int)blockIdx.x / a_tiles;
    int e, row0, rows, b0 = 0, red;
    if constexpr (OP == kOpDw) {
        const int n_tiles = (g.N + kSimTile - 1) / kSimTile;
        e = bt / n_tiles;
        b0 = (bt % n_tiles) * kSimTile;
        row0 = grouped_offset(g, e);
        rows = max(grouped_offset(g, e + 1) - row0, 0);
        red = rows;
    } else {
        const GroupedBlock b = grouped_find(grouped_scan(g, kSimTile), bt, kSimTile);
        if (b.e < 0) return;
        e = b.e;
        row0 = b.row0;
        rows = b.rows;
        red = OP == kOpFwd ? g.K : g.N;
    }
    const uint16_t* w = g.w + (size_t)e * g.N * g.K;
    const int b_rows = OP == kOpDw ? min(g.N - b0, kSimTile) : rows;

    f32x4_t acc[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) acc[v] = f32x4_t{0, 0, 0, 0};
    for (int r0 = 0; r0 < red; r0 += kSimStep) {
        // Element (i, r) of each tile; consecutive threads take consecutive
        // elements of the operand's contiguous dimension.
#pragma unroll
        for (int q = 0; q < kSimTile * kSimStep / 256; ++q) {
            const int t = q * 256 + tid;
            // operand A: reduction-contiguous for fwd, output-contiguous else
            {
                const int i = OP == kOpFwd ? t / kSimStep : t % kSimTile;
                const int r = OP == kOpFwd ? t % kSimStep : t / kSimTile;
                uint16_t v = 0;
                if (a0 + i < a_dim && r0 + r < red) {
                    if constexpr (OP == kOpFwd) {
                        v = w[(size_t)(a0 + i) * g.K + r0 + r];
                    } else if constexpr (OP == kOpDx) {
                        v = w[(size_t)(r0 + r) * g.K + a0 + i];
                    } else {
                        const int row = grouped_row(g, row0 + r0 + r, g.how_x);
                        if (row >= 0) v = g.x[(size_t)row * g.K + a0 + i];
                    }
                }
                la[i * kSimRow + r] = v;
            }
            {
                const int j = OP == kOpDw ? t % kSimTile : t / kSimStep;
                const int r = OP == kOpDw ? t / kSimTile : t % kSimStep;
                uint16_t v = 0;
                if (j < b_rows && r0 + r < red) {
                    if constexpr (OP == kOpDw) {
                        const int row = grouped_row(g, row0 + r0 + r, g.how_dy);
                        if (row >= 0) v = g.dy[(size_t)row * g.N + b0 + j];
                    } else {
                        const int row = grouped_row(g, row0 + j, OP == kOpFwd ? g.how_x : g.how_dy);
                        if (row >= 0)
                            v = (OP == kOpFwd ? g.x : g.dy)[(size_t)row * red + r0 + r];
                    }
                }
                lb[j * kSimRow + r] = v;
            }
        }
        __syncthreads();
        const int li = lane & 15, q = lane >> 4;
        const bf16x8_t fb = *reinterpret_cast<const bf16x8_t*>(&lb[(wave * 16 + li) * kSimRow + 8 * q]);
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            const bf16x8_t fa = *reinterpret_cast<const bf16x8_t*>(&la[(a * 16 + li) * kSimRow + 8 * q]);
            acc[a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa, fb, acc[a], 0, 0, 0);
        }
        __syncthreads();
    }
    // column j = wave*16 + lane%16 of B, rows a*16 + 4*(lane/16) + v of A
    const int j = wave * 16 + (lane & 15);
    if (j >= b_rows) return;
    size_t dst;
    if constexpr (OP == kOpDw) {
        dst = ((size_t)e * g.N + b0 + j) * g.K;
    } else {
        int row = row0 + j;
        if (g.how_out == kRowSlot) {
            row = grouped_row(g, row, kRowSlot);
            if (row < 0) return;
        }
        dst = (size_t)row * a_dim;
    }
#pragma unroll
    for (int a = 0; a < 4; ++a)
#pragma unroll
        for (int v = 0; v < 4; ++v) {
            const int c = a0 + a * 16 + 4 * (lane >> 4) + v;
            if (c >= a_dim) continue;
            if (g.out_f32) {
                float* o = (float*)g.out + dst + c;
                *o = g.accumulate ? *o + acc[a][v] : acc[a][v];
            } else {
                ((uint16_t*)g.out)[dst + c] = f32_to_bf16_bits(acc[a][v]);
            }
        }
}

int blocks_bound(const GroupedArgs& g, int B) {
    return g.R / B + (g.R < g.E ? g.R : g.E);
}

template <int OP>
void launch_any(const GroupedArgs& g, hipStream_t s) {
    const int a_tiles = ((OP == kOpFwd ? g.N : g.K) + kSimTile - 1) / kSimTile;
    const int b_tiles = OP == kOpDw ? g.E * ((g.N + kSimTile - 1) / kSimTile)
                                    : blocks_bound(g, kSimTile);
    grouped_any_kernel<OP><<<a_tiles * b_tiles, 256, 0, s>>>(g);
}

}  // namespace

// full tiles: every row of an operand is whole 16-byte chunks
static bool tiles_fit(const GroupedArgs& g) { return g.K % 8 == 0 && g.N % 8 == 0; }

void launch_grouped_fwd(const GroupedArgs& g, hipStream_t s) {
    if (tiles_fit(g)) launch_grouped_tiles_fwd(g, s);
    else launch_any<kOpFwd>(g, s);
}
void launch_grouped_dx(const GroupedArgs& g, hipStream_t s) {
    if (tiles_fit(g)) launch_grouped_tiles_dx(g, s);
    else launch_any<kOpDx>(g, s);
}
size_t grouped_dw_workspace(const GroupedArgs&) { return 0; }
void launch_grouped_dw(const GroupedArgs& g, void*, hipStream_t s) {
    if (tiles_fit(g)) launch_grouped_tiles_dw(g, s);
    else launch_any<kOpDw>(g, s);
}

}  // namespace moe
