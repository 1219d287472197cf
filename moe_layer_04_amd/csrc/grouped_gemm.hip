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
#include "../../include/moe.h"
#include "ckpt.hpp"
#include "grouped.hpp"
#include "small_tiles.hpp"
#include "tiles.hpp"

#include <type_traits>

namespace moe {

namespace {

constexpr int kOpFwd = 0, kOpDx = 1, kOpDw = 2;

// ---------------------------------------------------------------------------
// Small tiles, any widths: 64 x 64 outputs per workgroup of four waves (32 x 32
// each, 16x16x32 MFMAs), 64 reduction elements a step.  For products with too
// few outputs for 256 x 256 tiles, where the time is the latency of a step, and
// for rows that are not whole 16-byte chunks, which the copies of those tiles
// cannot take; for many outputs of such rows also as 128 x 128 (see wide).  A
// step's chunks of 8 elements are loaded into registers two steps ahead (16
// bytes at any 2-byte address; a row's last chunk as the row's last 8 elements,
// so that nothing past a row is read) and stored to one of two LDS buffers, a
// barrier a step.
//
// LDS layouts: small_tiles.hpp.
//
// 16x16x32: lane l supplies row l % 16, reduction 8*(l/16)..+8; its
// accumulators are rows 4*(l/16)+v of column l % 16.
//
// Bound by the latency of a step, 0.5-0.6 us with up to two workgroups a CU
// (1024 rows of one expert, 4096 -> 1024: 34.9 us for 64 steps).  406 rows over 7
// experts of 1001 x 330, dx: 11.5 us a call of 16 steps; 666 rows over 8 experts,
// dw of 1032 x 256 in fp32: 7.5 us.
// ---------------------------------------------------------------------------
constexpr int kSimAhead = 2;                   // steps loaded ahead

// The tile of a weight gradient, `rows` x `cols` values of it from `first` on,
// through LDS: a store instruction writes whole rows of the tile, where the
// accumulators hold 16 rows of four values (16 rows over 8 experts of 1433 x 4095:
// 32.7 us against 57.4; 4096 rows, 4097 x 2049 in bf16: 181 against 221).  Chunks of 16
// bytes are permuted by the row.
template <int TILE, bool F32>
__device__ __forceinline__ void store_grad(char* lds, const f32x4_t (&acc)[TILE / 32][TILE / 32],
                                           const GroupedArgs& g, size_t first, int rows, int cols,
                                           int fa0, int fb0) {
    constexpr int size = F32 ? 4 : 2, per = 16 / size, chunks = TILE / per;
    const int lane = lane_id();
    auto at = [](int row, int chunk) { return row * TILE * size + ((chunk ^ (row & 7)) << 4); };
    __syncthreads();  // the last step's fragments are read
#pragma unroll
    for (int b = 0; b < TILE / 32; ++b)
#pragma unroll
        for (int a = 0; a < TILE / 32; ++a) {
            const int row = fb0 + 16 * b + (lane & 15), col = fa0 + 16 * a + 4 * (lane >> 4);
            const f32x4_t v = acc[a][b];
            if constexpr (F32)
                *reinterpret_cast<f32x4_t*>(lds + at(row, col / per)) = v;
            else
                *reinterpret_cast<uint2*>(lds + at(row, col / per) + (col & 4) * 2) =
                    uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        }
    __syncthreads();
    typedef typename std::conditional<F32, f32x4_t, u16x8_t>::type chunk_t;
    typedef typename std::conditional<F32, float, uint16_t>::type value_t;
    typedef chunk_t any_t __attribute__((aligned(size)));
#pragma unroll 4
    for (int i = (int)threadIdx.x; i < TILE * chunks; i += 256) {
        const int row = i / chunks, c = i % chunks;
        if (row >= rows || c * per >= cols) continue;
        chunk_t v = *reinterpret_cast<const chunk_t*>(lds + at(row, c));
        value_t* o = (value_t*)g.out + first + (size_t)row * g.K + c * per;
        if (c * per + per <= cols) {
            any_t* p = reinterpret_cast<any_t*>(o);
            if constexpr (F32) {
                if (g.accumulate) v += *p;
            }
            *p = v;
        } else {
#pragma unroll
            for (int j = 0; j < per - 1; ++j)
                if (c * per + j < cols) o[j] = F32 && g.accumulate ? o[j] + v[j] : v[j];
        }
    }
}

// A chunk of x kept in 8 bits, loaded and settled as one of bf16 (load_chunk); its
// values are formed when it is stored.
struct KeptChunk {
    u32x2_t codes;
    uint32_t X;
};
template <Widths W>
__device__ __forceinline__ KeptChunk load_kept(const GroupedArgs& g, int row, int c) {
    const bool in = row >= 0 && c < g.K;
    const int8_t* zeros = reinterpret_cast<const int8_t*>(kZeros);
    const int8_t* codes = in ? g.codes + (size_t)row * g.K : zeros;
    const uint8_t* scale = in ? g.scales + (size_t)row * ckpt_blocks(g.K) + c / kCkptBlock
                              : reinterpret_cast<const uint8_t*>(zeros);
    typedef const __attribute__((address_space(1))) uint8_t* global_scale_t;
    KeptChunk v;
    v.X = *(global_scale_t)(uintptr_t)scale;
    if constexpr (W == Widths::kWhole) {
        typedef const __attribute__((address_space(1))) u32x2_t* global_t;
        v.codes = *(global_t)(uintptr_t)(codes + (in ? c : 0));
    } else if (W == Widths::kAny && g.K < 8) {
        uint64_t b = 0;
#pragma unroll
        for (int i = 0; i < 7; ++i)
            if (in && c + i < g.K) b |= (uint64_t)(uint8_t)codes[c + i] << (8 * i);
        v.codes = __builtin_bit_cast(u32x2_t, b);
    } else {
        typedef const __attribute__((address_space(1))) u32x2_any_t* global_t;
        v.codes = *(global_t)(uintptr_t)(codes + (in ? min(c, g.K - 8) : 0));
    }
    return v;
}
using moe::settle_chunk;
__device__ __forceinline__ KeptChunk settle_chunk(KeptChunk v, int c, int width) {
    const int by = width < 8 ? 0 : min(max(c - (width - 8), 0), 7);  // (8 and more: no columns, zeros)
    v.codes = __builtin_bit_cast(u32x2_t, __builtin_bit_cast(uint64_t, v.codes) >> (8 * by));
    return v;
}
__device__ __forceinline__ u16x8_t chunk_bits(u16x8_t v) { return v; }
__device__ __forceinline__ u16x8_t chunk_bits(KeptChunk v) {
    float f[V];
    ckpt_values(v.codes, v.X, f);
    const uint4 w = {pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                     pack_bf16x2(f[6], f[7])};
    return __builtin_bit_cast(u16x8_t, w);
}

template <int OP, Widths W, int TILE, bool KEPT>
__global__ __launch_bounds__(256, TILE > kSim || KEPT ? 2 : OP == kOpDw ? 3 : 4) void grouped_small_kernel(
    GroupedArgs g) {
    constexpr bool ACOL = OP != kOpFwd, BCOL = OP == kOpDw;
    constexpr int AHEAD = TILE > kSim && OP == kOpDw ? 1 : kSimAhead;
    constexpr int SUBS = TILE / kSim, H = 2 * SUBS, F = TILE / 32;  // parts, chunks and fragments of an operand
    constexpr int kOperand = SUBS * kSimBytes;
    __shared__ __attribute__((aligned(16))) char lds[2][2 * kOperand];
    const int tid = (int)threadIdx.x, lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int a_dim = OP == kOpFwd ? g.N : g.K;
    const int a_tiles = (a_dim + TILE - 1) / TILE;
    int tile = (int)blockIdx.x;
    // Where rows of the output (and of dx's weights) are no whole lines of 128
    // bytes, neighbouring tiles share lines: they go to one XCD (workgroup g runs
    // on XCD g % 8), whose L2 joins them.  dw, us: 4 rows over 99 experts of 8768
    // x 1042 in fp32 1409 apart, 572 so; dx 8x2/8 14337 -> 4095 220, 198; whole
    // lines, dw 1024/8 1024 x 1024: 13.6, 14.6; fwd 64x2/8 4095 -> 14337: 228, 257.
    if (OP != kOpFwd && (uint32_t)a_dim * (OP == kOpDw && g.out_f32 ? 4 : 2) % 128 != 0) {
        const int per_xcd = (int)gridDim.x / 8;
        tile = tile % 8 * per_xcd + tile / 8;
    }
    const int a0 = (tile % a_tiles) * TILE;  // first output column
    int bt = tile / a_tiles, sp = 0;
    int e, row0, rows, b0 = 0, red;
    if constexpr (OP == kOpDw) {
        const int n_tiles = (g.N + TILE - 1) / TILE;
        e = bt / n_tiles;
        if (e >= g.E) return;  // the grid is rounded up
        b0 = (bt % n_tiles) * TILE;
        row0 = grouped_offset_scalar(g, e);
        rows = max(grouped_offset_scalar(g, e + 1) - row0, 0);
        red = rows;
        if (rows == 0 && g.accumulate) return;
    } else {
        sp = bt % g.splits;
        bt /= g.splits;
        const GroupedBlock b = grouped_find(grouped_scan(g, TILE), bt, TILE);
        if (b.e < 0) return;
        e = b.e;
        row0 = b.row0;
        rows = b.rows;
        red = OP == kOpFwd ? g.K : g.N;
    }
    const uint16_t* w = g.w + (size_t)e * g.N * g.K;
    const int b_rows = OP == kOpDw ? min(g.N - b0, TILE) : rows;

    // this thread's chunks of an operand: c of rows r + 32h, or, where the rows
    // run along the reduction, c of the h/2-th 64 columns of rows r and r + 32
    const int r = tid >> 3, c = tid & 7;
    auto col_row = [&](int h) { return r + 32 * (h & 1); };
    auto col_at = [&](int h) { return (h >> 1) * kSim + c * 8; };
    const int fa0 = (wave & 1) * (TILE / 2), fb0 = (wave >> 1) * (TILE / 2);
    const uint16_t* brow[H];  // fwd, dx: fixed rows of B
    if constexpr (OP != kOpDw) {
#pragma unroll
        for (int h = 0; h < H; ++h) {
            brow[h] = nullptr;
            const int j = r + 32 * h;
            const int row = j < rows ? grouped_row(g, row0 + j, OP == kOpFwd ? g.how_x : g.how_dy) : -1;
            if (row >= 0) brow[h] = (OP == kOpFwd ? g.x : g.dy) + (size_t)row * red;
        }
    }
    typedef typename std::conditional<KEPT, KeptChunk, u16x8_t>::type chunk_a_t;
    struct Step {
        chunk_a_t a[H];
        u16x8_t b[H];
    };
    auto load = [&](int step) {
        Step s;
        const int r0 = step * kSim;
        if constexpr (OP == kOpDw) {
            int rx[2], ry[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int at = r0 + col_row(i);
                rx[i] = ry[i] = -1;
                if (at < red) {
                    rx[i] = ry[i] = row0 + at;
                    if (g.sorted) {  // one slot for both operands' rows
                        const uint32_t p = (uint32_t)g.sorted[row0 + at];
                        const int t = (int)grouped_token(p, g.magic);
                        rx[i] = p >= g.slots ? -1 : g.how_x == kRowToken ? t : rx[i];
                        ry[i] = p >= g.slots ? -1 : g.how_dy == kRowToken ? t : ry[i];
                    }
                }
            }
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const int x = rx[h & 1], y = ry[h & 1];
                if constexpr (KEPT) s.a[h] = load_kept<W>(g, x, a0 + col_at(h));
                else s.a[h] = load_chunk<W>(x < 0 ? nullptr : g.x + (size_t)x * g.K, a0 + col_at(h), g.K);
                s.b[h] = load_chunk<W>(y < 0 ? nullptr : g.dy + (size_t)y * g.N, b0 + col_at(h), g.N);
            }
        } else {
#pragma unroll
            for (int h = 0; h < H; ++h) {
                if constexpr (OP == kOpFwd) {
                    const int n = a0 + r + 32 * h;
                    s.a[h] = load_chunk<W>(n < g.N ? w + (size_t)n * g.K : nullptr, r0 + c * 8, red);
                } else {
                    const int n = r0 + col_row(h);
                    s.a[h] = load_chunk<W>(n < red ? w + (size_t)n * g.K : nullptr, a0 + col_at(h), g.K);
                }
                s.b[h] = load_chunk<W>(brow[h], r0 + c * 8, red);
            }
        }
        return s;
    };
    // whether a step has chunks to settle: last columns of the tile, or the end
    // of a reduction that runs along the rows
    const bool a_ends = ACOL && a0 + TILE > g.K, b_ends = BCOL && b0 + TILE > g.N;
    auto settle = [&](Step& s, int step) {
        if constexpr (W == Widths::kWhole) return;
        const int r0 = step * kSim;
        if (a_ends || (!ACOL && r0 + kSim > red)) {
#pragma unroll
            for (int h = 0; h < H; ++h)
                s.a[h] = settle_chunk(s.a[h], ACOL ? a0 + col_at(h) : r0 + c * 8, ACOL ? g.K : red);
        }
        if (b_ends || (!BCOL && r0 + kSim > red)) {
#pragma unroll
            for (int h = 0; h < H; ++h)
                s.b[h] = settle_chunk(s.b[h], BCOL ? b0 + col_at(h) : r0 + c * 8, BCOL ? g.N : red);
        }
    };
    f32x4_t acc[F][F];
#pragma unroll
    for (int a = 0; a < F; ++a)
#pragma unroll
        for (int b = 0; b < F; ++b) acc[a][b] = f32x4_t{0, 0, 0, 0};
    int first = 0, steps = (red + kSim - 1) / kSim;
    if constexpr (OP != kOpDw) {
        const GroupedRange range = grouped_range(steps, g.splits, sp);
        first = range.first;
        steps = range.count;
    }
    Step ahead[AHEAD];
#pragma unroll
    for (int i = 0; i < AHEAD; ++i)
        if (i < steps) ahead[i] = load(first + i);
    for (int s0 = 0; s0 < steps; s0 += AHEAD) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) {
            const int s = s0 + i;
            if (s >= steps) break;
            char* buf = lds[s & 1];
            settle(ahead[i], first + s);
#pragma unroll
            for (int h = 0; h < H; ++h) {
                // the h/2-th 64 rows or columns
                char* to = buf + (h >> 1) * kSimBytes;
                *reinterpret_cast<u16x8_t*>(to + sim_at<ACOL>(col_row(h), c)) = chunk_bits(ahead[i].a[h]);
                *reinterpret_cast<u16x8_t*>(to + kOperand + sim_at<BCOL>(col_row(h), c)) = ahead[i].b[h];
            }
            // the buffer written next was last read before this barrier
            __syncthreads();
            if (s + AHEAD < steps) ahead[i] = load(first + s + AHEAD);
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                bf16x8_t fa[F], fb[F];
                const char* pa = buf + fa0 / kSim * kSimBytes;
                const char* pb = buf + kOperand + fb0 / kSim * kSimBytes;
#pragma unroll
                for (int f = 0; f < F; ++f) {
                    fa[f] = sim_frag<ACOL>(pa, fa0 % kSim + 16 * f, ks, lane);
                    fb[f] = sim_frag<BCOL>(pb, fb0 % kSim + 16 * f, ks, lane);
                }
#pragma unroll
                for (int a = 0; a < F; ++a)
#pragma unroll
                    for (int b = 0; b < F; ++b)
                        acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[a], fb[b], acc[a][b], 0, 0, 0);
            }
        }
    }
    if constexpr (OP == kOpDw) {
        const size_t at = ((size_t)e * g.N + b0) * g.K + a0;
        const int cols = min(g.K - a0, TILE);
        if (g.out_f32) store_grad<TILE, true>(lds[0], acc, g, at, b_rows, cols, fa0, fb0);
        else store_grad<TILE, false>(lds[0], acc, g, at, b_rows, cols, fa0, fb0);
        return;
    }
    // Padding rows are looked for only where a sum is NaN: finite weights leave
    // them zeros (looked for before the loop the smallest calls took 0.2 us more of
    // 5 to 10; so 0.1)
    bool nan = false;
#pragma unroll
    for (int a = 0; a < F; ++a)
#pragma unroll
        for (int b = 0; b < F; ++b) {
            const f32x4_t v = acc[a][b];
            nan |= __builtin_isunordered(v[0], v[1]) | __builtin_isunordered(v[2], v[3]);
        }
    if (__builtin_expect(__any(nan), 0)) {
        const uint64_t padding = grouped_padding(g, row0, rows, fb0);
#pragma unroll
        for (int b = 0; b < F; ++b)
            if (padding >> (16 * b + (lane & 15)) & 1) {
#pragma unroll
                for (int a = 0; a < F; ++a) acc[a][b] = f32x4_t{0, 0, 0, 0};
            }
    }
#pragma unroll
    for (int b = 0; b < F; ++b) {
        const int j = fb0 + 16 * b + (lane & 15);
        if (j >= b_rows) continue;
        int row = row0 + j;
        if (g.splits == 1 && g.how_out == kRowSlot) {
            row = grouped_row(g, row, kRowSlot);
            if (row < 0) continue;
        }
#pragma unroll
        for (int a = 0; a < F; ++a) {
            const int col = a0 + fa0 + 16 * a + 4 * (lane >> 4);
            const f32x4_t v = acc[a][b];
            if (g.splits > 1) {
                if (col < a_dim)
                    *reinterpret_cast<f32x4_t*>((float*)g.out + ((size_t)sp * g.R + row0 + j) *
                                                grouped_part_ld(a_dim) + col) = v;
            } else {
                uint16_t* o = (uint16_t*)g.out + (size_t)row * a_dim + col;
                u16x4_t q;
#pragma unroll
                for (int i = 0; i < 4; ++i) q[i] = f32_to_bf16_bits(v[i]);
                if (col + 4 <= a_dim) {
                    *reinterpret_cast<u16x4_any_t*>(o) = q;
                } else {
#pragma unroll
                    for (int i = 0; i < 3; ++i)
                        if (col + i < a_dim) o[i] = q[i];
                }
            }
        }
    }
}

int blocks_bound(const GroupedArgs& g, int B) {
    return g.R / B + (g.R < g.E ? g.R : g.E);
}

// every row of an operand is whole 16-byte chunks
bool chunked(const GroupedArgs& g) { return g.K % 8 == 0 && g.N % 8 == 0; }

int small_workgroups(const GroupedArgs& g, int op, int tile) {
    const int a_tiles = ((op == kOpFwd ? g.N : g.K) + tile - 1) / tile;
    const int b_tiles = op == kOpDw ? g.E * ((g.N + tile - 1) / tile) : blocks_bound(g, tile) * g.splits;
    return (a_tiles * b_tiles + 7) / 8 * 8;
}
template <int OP, Widths W, int TILE>
void launch_small_tiles(const GroupedArgs& g, hipStream_t s) {
    const int grid = small_workgroups(g, OP, TILE);
    if constexpr (OP == kOpDw && TILE == kSim) {
        if (g.codes) {
            grouped_small_kernel<OP, W, TILE, true><<<grid, 256, 0, s>>>(g);
            return;
        }
    }
    grouped_small_kernel<OP, W, TILE, false><<<grid, 256, 0, s>>>(g);
}
// Rows that are no whole chunks, with enough of them and enough outputs, on 128
// x 128 tiles: half the loads an output.  us, 64 / 128, T tokens x k over E
// experts (128 x 128 tiles):
//   fwd K->N  2048x2/8 2049->4097 [1056] 227/166, 1000x1/1 4095->4097 [264] 123/94,
//             512x2/8 1025->4097 [264] 43.2/38.4, 1025->2049 [136] 26.3/27.8;
//             8x2/8 4095->14337 [904, two rows an expert] 176/192
//   dx  N->K  2048x2/8 4097->2049 [544] 294/203, 512x2/8 1433->4095 [256] 53.7/48.1,
//             4097->1025 [72] 59/89
//   dw  N x K, rows looked up, an even routing, bf16 and fp32: 2048x2/8 4097x2049 [4488]
//             302/166 and 336/206, 4096x2/8 1025x1025 [648] 92/64 and 90/63, 513x513
//             [200] 26.6/29.8 and 27.5/31.1, 512x2/8 1025x1025 [648] 20.2/16.8 and 22.7/19.2
bool wide(const GroupedArgs& g, int op) {
    if (chunked(g) || g.K < 8 || g.N < 8) return false;
    const auto tiles = [](int width) { return (long)((width + 2 * kSim - 1) / (2 * kSim)); };
    if (op == kOpDw) return g.E * tiles(g.N) * tiles(g.K) >= 512;
    const long experts = g.R < g.E ? g.R : g.E, blocks = tiles(g.R);
    return g.R >= kSim * experts && tiles(op == kOpFwd ? g.N : g.K) * (blocks > experts ? blocks : experts) >= 256;
}
template <int OP>
void launch_small(const GroupedArgs& g, hipStream_t s) {
    if (chunked(g)) launch_small_tiles<OP, Widths::kWhole, kSim>(g, s);
    else if (g.K < 8 || g.N < 8) launch_small_tiles<OP, Widths::kAny, kSim>(g, s);
    else if (wide(g, OP)) launch_small_tiles<OP, Widths::kLong, 2 * kSim>(g, s);
    else launch_small_tiles<OP, Widths::kLong, kSim>(g, s);
}

}  // namespace

namespace {
// y = the ranges' products added up in order, a thread per four values; row i
// goes where the product would have put it
__global__ __launch_bounds__(256) void rows_join_kernel(const float* __restrict__ parts, GroupedArgs g,
                                                        int width) {
    const int ld = grouped_part_ld(width);
    const uint32_t at = blockIdx.x * 256u + threadIdx.x;
    const int i = (int)(at / (uint32_t)(ld / 4)), col = (int)(at % (uint32_t)(ld / 4)) * 4;
    if (i >= g.R || i < grouped_offset(g, 0) || i >= grouped_offset(g, g.E)) return;
    const int row = g.how_out == kRowSlot ? grouped_row(g, i, kRowSlot) : i;
    if (row < 0) return;
    const float* p = parts + (size_t)i * ld + col;
    const size_t next = (size_t)g.R * ld;
    f32x4_t v = *reinterpret_cast<const f32x4_t*>(p);
#pragma unroll 4
    for (int s = 1; s < g.splits; ++s) v += *reinterpret_cast<const f32x4_t*>(p + s * next);
    uint16_t* o = (uint16_t*)g.out + (size_t)row * width + col;
    u16x4_t q;
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = f32_to_bf16_bits(v[j]);
    if (col + 4 <= width) {
        *reinterpret_cast<u16x4_any_t*>(o) = q;
    } else {
#pragma unroll
        for (int j = 0; j < 3; ++j)
            if (col + j < width) o[j] = q[j];
    }
}

// How a rows product is computed: on which tiles, and in how many ranges of its
// reduction.  us; (tokens x k / experts, reduction -> columns).
//
// The weight stream (forward) while an expert has up to three rows on average.
// Stream / best of the tiles: 1x2/16 4096->16384 40/42, 8x2/8 4096->28672
// 286/317, 1x1/1 4096->4096 11.1/13.1; at four rows 16x2/8 4096->28672 317/324
// and 128x8/256 2048->7168 1277/1257, at eight 32x2/8 4096->28672 339/324.  In
// ranges up to a workgroup a CU, if a wave has 32 steps or more to share:
// 1x6/21 10328->272 18.9 whole, 13.5 in four; 1x1/1 14336->4096 30.7, 22.1 in
// two, but 1x1/1 4096->4096 11.1, 13.7 in two (the second launch).
//
// Full tiles above 512 small ones, or fewer with so many steps that ranges of
// them fill the chip.  Small / full, each in its best number of ranges:
//   fwd 512x2/8   1024->2048 16.3/21.9,   4096->2048 49.8/40.7,  14336->2048 188/114
//       1024x1/1  1024->1024 9.9/22.4,    4096->1024 25.2/29.9,  14336->1024 62.9/46.3
//                 1024->4096 19.8/23.3,   2048->4096 33.8/36.6,  4096->4096 63.1/49.2
//   dx  2048x2/8  1024->512 17.7/24.4,    2048->512 29.5/29.0,   14336->512 186/89
//                 1024->1024 28.5/25.4,   4096->1024 85.1/53.7
//       37x8/8    14336->512 33.9/33.3,   14336->1024 49.2/44.0, 14336->2048 102/93
//       8x2/8     28672->4096 313/269;    8192x2/8 512->256 19.2/16.5
// but small ones for short reductions of experts with few rows, where a full
// tile is mostly its start and end:
//   fwd 160x8/128 64->4096 22.7/43.0, 192->8192 85/130, 512->4096 98/118,
//                 2048->2048 223/188;  640x8/128 512->4096 119/131;
//       1280x8/128 64->4096 56.1/51.3, 512->4096 174/145
//   dx  128x8/128 64->4096 24.8/43.8, 192->8192 92/124, 512->4096 110/127,
//                 1024->2048 110/104;  640x8/128 512->4096 136/136
//
// Ranges of full tiles while a CU has no more than one and a range 16 steps:
// 1024x1/1 14336->1024 214 whole, 68.6 in four, 46.3 in eight; 4096->4096 67.1,
// 51.4, 49.2 (two, four); two ranges of 8 steps 1024->4096 23.3, 29.6.  Of small
// tiles up to 2.5 a CU, while a range has eight steps and the whole 32:
// 1024x1/1 4096->512 34.9 whole, 18.7 in four, 21.1 in eight; 2048->512 19.4,
// 13.7, 16.1; 1024->512 9.8, 13.4 (four).
struct RowsPlan {
    enum { kStream, kFull, kSmall } on;
    int splits;
};
RowsPlan rows_plan(const GroupedArgs& g, bool dx) {
    const int cols = dx ? g.K : g.N;
    const long steps = ((dx ? g.N : g.K) + 63) / 64;  // of either tiles and of the stream
    const long experts = g.R < g.E ? g.R : g.E;
    const long small_blocks = g.R / kSim, full_blocks = g.R / 256 + experts / 2;
    const long small = (long)((cols + 63) / 64) * (small_blocks > experts ? small_blocks : experts);
    const long full = (long)((cols + 255) / 256) * (full_blocks > experts ? full_blocks : experts);
    RowsPlan p = {RowsPlan::kSmall, 1};
    if (chunked(g) && !dx && g.R <= 3 * experts) p.on = RowsPlan::kStream;
    else if (chunked(g) && (small > 512 || small * steps >= 512 * 64) &&
             (steps > 8 || g.R > 48 * experts))
        p.on = RowsPlan::kFull;
    long work, most, least;  // workgroups whole, the most of them, a range's least steps
    if (p.on == RowsPlan::kStream) {
        work = (long)((cols + 31) / 32) * experts;
        most = 256;
        least = steps < 128 ? steps : 32;
    } else if (p.on == RowsPlan::kFull) {
        work = full;
        most = 256;
        least = 16;
    } else {
        work = small;
        most = 640;
        least = steps < 32 ? steps : 8;
    }
    while (p.splits < 16 && work * p.splits * 2 <= most && steps / (p.splits * 2) >= least) p.splits *= 2;
    return p;
}

size_t rows_workspace(const GroupedArgs& g, bool dx) {
    if (g.R == 0) return 0;
    const int splits = rows_plan(g, dx).splits;
    return splits > 1 ? (size_t)splits * g.R * grouped_part_ld(dx ? g.K : g.N) * 4 : 0;
}

template <bool DX>
void launch_rows(const GroupedArgs& call, void* workspace, hipStream_t s) {
    GroupedArgs g = call;
    const RowsPlan plan = rows_plan(g, DX);
    g.splits = plan.splits;
    if (g.splits > 1) g.out = workspace;
    if (plan.on == RowsPlan::kStream) launch_grouped_stream_fwd(g, s);
    else if (plan.on == RowsPlan::kSmall) launch_small<DX ? kOpDx : kOpFwd>(g, s);
    else if (DX) launch_grouped_tiles_dx(g, s);
    else launch_grouped_tiles_fwd(g, s);
    if (g.splits > 1) {
        const int width = DX ? g.K : g.N;
        const long threads = (long)g.R * (grouped_part_ld(width) / 4);
        g.out = call.out;
        rows_join_kernel<<<(int)((threads + 255) / 256), 256, 0, s>>>((const float*)workspace, g, width);
    }
}

// The weight gradient on small or on full tiles, by an estimate of what they
// take in 1/20 us a CU: 11 a step of a small tile (with its share of a CU's four)
// and 3 to store it; 29 a step of a full tile, 64 to store it and 100 to start.
// us, small / full, rows over E experts of N x K (small tiles, steps):
//   1024/8 1024x1024 [2048, 2] 13.5/14.4    2048/8 the same [4] 22.2/17.2
//   4096/8 1024x256 [512, 8] 14.7/21.0      8192/8 the same [16] 26.2/29.2
//   16384/8 the same [32] 47.4/32.5         512/8 2048x1024 [4096, 1] 20.0/13.1
//   256/8 4096x4096 [32768, 1] 88.5/57.5    19/38 2056x128 [2508, 1] 10.0/21.4
//   54/73 64x5696 [6497, 1] 17.9/35.3       488/245 576x192 [6615, 1] 21.2/29.7
//   4096/1 512x512 [64, 64] 47.2/24.0       7448/12 128x3032 [1152, 10] 30.8/22.3
bool small_dw(const GroupedArgs& g) {
    if (!chunked(g) || g.R == 0) return true;
    const long experts = g.R < g.E ? g.R : g.E, steps = (g.R / experts + kSim - 1) / kSim;
    auto tiles = [&](int side) { return (long)((g.K + side - 1) / side) * ((g.N + side - 1) / side) * g.E; };
    const long small = tiles(kSim) > 256 ? tiles(kSim) : 256;
    const int splits = grouped_tiles_dw_splits(g);
    const long rounds = (tiles(256) * splits + 255) / 256, part = (steps + splits - 1) / splits;
    return small * (11 * steps + 3) <= 256 * (rounds * (29 * part + 64) + 100);
}
}  // namespace

GroupedPlan grouped_plan(const GroupedArgs& call, int op) {
    static_assert(kOpFwd == MOE_PRODUCT_FWD && kOpDx == MOE_PRODUCT_DX && kOpDw == MOE_PRODUCT_DW, "");
    if (op != kOpDw && call.R == 0) return {MOE_PRODUCT_TILES_64, 1, 0};  // nothing is launched
    GroupedArgs g = call;
    bool stream = false, small;
    if (op == kOpDw) {
        small = small_dw(g);
        g.splits = small ? 1 : grouped_tiles_dw_splits(g);
    } else {
        const RowsPlan p = rows_plan(g, op == kOpDx);
        stream = p.on == RowsPlan::kStream;
        small = p.on == RowsPlan::kSmall;
        g.splits = p.splits;
    }
    if (stream) return {MOE_PRODUCT_STREAM, g.splits, grouped_stream_workgroups(g)};
    if (small) {
        const int tile = wide(g, op) ? 2 * kSim : kSim;
        return {tile > kSim ? MOE_PRODUCT_TILES_128 : MOE_PRODUCT_TILES_64, g.splits,
                small_workgroups(g, op, tile)};
    }
    return {MOE_PRODUCT_TILES_256, g.splits,
            op == kOpDw ? grouped_tiles_dw_workgroups(g) : grouped_tiles_rows_workgroups(g, op == kOpDx)};
}

size_t grouped_fwd_workspace(const GroupedArgs& g) { return rows_workspace(g, false); }
size_t grouped_dx_workspace(const GroupedArgs& g) { return rows_workspace(g, true); }
void launch_grouped_fwd(const GroupedArgs& g, void* workspace, hipStream_t s) {
    launch_rows<false>(g, workspace, s);
}
void launch_grouped_dx(const GroupedArgs& g, void* workspace, hipStream_t s) {
    launch_rows<true>(g, workspace, s);
}

size_t grouped_dw_workspace(const GroupedArgs& g) {
    const int splits = small_dw(g) ? 1 : grouped_tiles_dw_splits(g);
    return splits > 1 ? (size_t)splits * g.E * g.N * g.K * 4 : 0;
}
// x kept in 8 bits: few small tiles form its values as they store them to LDS, each
// its own; with more of them a launch that brings the rows back costs less.  us a
// call, so / brought back (the same in a captured graph), rows / experts, N x K
// [tiles, steps]:
//   666/8 1032x256 [544, 2] 11.2/15.1 (8.8/8.6), 1000/7 1001x330 [672, 3] 11.6/15.1
//   (9.1/11.4), 1024/8 1024x512 [1024, 2] 17.2/21.7 (12.5/12.4), 1024x640 [1280, 2]
//   16.0/20.8 (15.5/14.7), 1024x768 [1536, 2] 17.6/21.5 (17.7/15.1), 1024x1024 [2048, 2]
//   21.5/17.8 (21.9/18.2); 512/1 512x512 [64, 8] 11.7/14.7 (11.7/12.9), 8192/8 513x513
//   [648, 16] 30.8/33.7, 8192/4 1001x1001 [1024, 32] 73/101, 2048/1 [256, 32] 41/50
// A hundred steps and more would take the launch as well, which this rule leaves out:
//   8192/1 1001x1001 [256, 128] 198/176, 509x509 [64, 128] 202/181, 32768/1 333x333
//   [36, 512] 827/736
// (128 x 128 tiles read bf16 only: 4096/8 4097x2049 356 with codes, 320.)
bool grouped_dw_restores(const GroupedArgs& g) {
    return !small_dw(g) || wide(g, kOpDw) || small_workgroups(g, kOpDw, kSim) > 1024;
}
void launch_grouped_dw(const GroupedArgs& call, void* workspace, hipStream_t s) {
    GroupedArgs g = call;
    if (small_dw(g)) {
        launch_small<kOpDw>(g, s);
    } else {
        g.splits = grouped_tiles_dw_splits(g);
        launch_grouped_tiles_dw(g, workspace, s);
    }
}

}  // namespace moe
