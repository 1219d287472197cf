// grouped_stream.hip -- the grouped forward product for very few rows an expert
// (decoding): the weights of the experts that have rows are read once and
// everything else is small, so the kernel is a stream of W through the matrix
// cores, bound by HBM reads.
//
// A workgroup of four waves takes 32 rows of W[e] against one block of up to 16
// rows of x, a quarter of the reduction a wave; of a short reduction 32 rows a
// wave (280 rows over 200 experts, us, quarters / whole: 15168 x 192 390/198,
// 4096 x 512 143/112, 4096 x 1024 226/213, but 512 x 1024 29.7/31.7).  No LDS in
// the main loop: a wave loads its fragments straight into registers, two steps
// ahead.
// 16x16x32 MFMA: lane l supplies row l % 16, reduction 8*(l/16)..+8, so a load
// instruction takes 64 bytes of each of 16 rows; a step is 64 reduction
// elements, 128 bytes a row.  x comes from L2 (a block's rows are read by every
// workgroup of its expert).  The waves' sums meet in LDS at the end, in wave
// order.  Every wave starts its quarter at another step: waves that walk it in
// step ask for one column of rows that lie K*2 bytes apart, few memory
// channels at a time.
//
// One token, two of 16 experts of 16384 x 4096 (268 MB), weights not in any
// cache, us: this kernel 49 (5.5 TB/s); walking in step 64; neighbouring steps
// to the four waves 51; three / four steps ahead 54 / 51; eight waves 54;
// 128-element steps 53; 64 x 64 tiles 57.  8 tokens x 2 over 8 experts of
// 28672 x 4096: 286 against 317 on full tiles.
//
// Reads are bounds-checked: rows past the end of W[e] or of the block, padding
// rows and the reduction's tail are offsets out of range, zeros without a
// memory access.
#include "grouped.hpp"
#include "tiles.hpp"

namespace moe {

namespace {

constexpr int kRowsA = 32, kRowsB = 16, kStep = 64, kWaves = 4, kAhead = 2;
constexpr int kWhole = 512;  // longest reduction that a wave takes whole

// QUARTERS: a wave takes a quarter of the reduction, else all of it for 32 rows
// of its own
template <bool QUARTERS>
__global__ __launch_bounds__(kWaves * 64) void grouped_stream_kernel(GroupedArgs g) {
    __shared__ f32x4_t part[QUARTERS ? kWaves - 1 : 1][2][64];
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    constexpr int kRowsGroup = QUARTERS ? kRowsA : kRowsA * kWaves;
    const int a_tiles = (g.N + kRowsGroup - 1) / kRowsGroup;
    const int bt = (int)blockIdx.x / a_tiles, sp = bt % g.splits;
    const GroupedBlock blk = grouped_find(grouped_scan(g, kRowsB), bt / g.splits, kRowsB);
    if (blk.e < 0) return;
    const int a0 = ((int)blockIdx.x % a_tiles) * kRowsGroup + (QUARTERS ? 0 : wave * kRowsA);
    if (!QUARTERS && a0 >= g.N) return;
    const uint32_t ld = (uint32_t)g.K * 2;
    const prsrc_t rw = pmake_rsrc(g.w + ((size_t)blk.e * g.N + a0) * g.K,
                                  (uint32_t)min(g.N - a0, kRowsA) * ld);
    const bool token = g.how_x == kRowToken;
    const prsrc_t rx = pmake_rsrc(token ? g.x : g.x + (size_t)blk.row0 * g.K,
                                  (uint32_t)(token ? g.T : blk.rows) * ld);
    const int li = lane & 15, q = lane >> 4;
    uint32_t woff[2], xoff = kNowhere;
#pragma unroll
    for (int a = 0; a < 2; ++a) woff[a] = (uint32_t)(16 * a + li) * ld + (uint32_t)(q * 16);
    if (li < blk.rows) {
        const int row = grouped_row(g, blk.row0 + li, g.how_x);
        if (row >= 0) xoff = (uint32_t)(token ? row : li) * ld + (uint32_t)(q * 16);
    }
    struct Frags { i32x4_t w[2][2], x[2]; };
    auto load = [&](int s) {
        Frags f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t kb = (uint32_t)(s * kStep + h * 32) * 2;
            const bool in = kb + (uint32_t)(q * 16) < ld;  // false past the last step too
#pragma unroll
            for (int a = 0; a < 2; ++a)
                f.w[a][h] = __builtin_amdgcn_raw_buffer_load_b128(rw, in ? woff[a] + kb : kNowhere, 0, 0);
            // kNowhere + kb is nowhere as well
            f.x[h] = __builtin_amdgcn_raw_buffer_load_b128(rx, in ? xoff + kb : kNowhere, 0, 0);
        }
        return f;
    };
    f32x4_t acc[2] = {};
    const int parts = QUARTERS ? kWaves * g.splits : 1, first = QUARTERS ? sp * kWaves + wave : 0;
    const int steps = (g.K + kStep - 1) / kStep, per = (steps + parts - 1) / parts;
    const int turn = ((int)blockIdx.x * 7 + wave * 3) % per;
    // the wave's s-th step; past its quarter: a step past the reduction
    auto step = [&](int s) {
        const int t = s + turn;
        return s < per ? first * per + (t < per ? t : t - per) : parts * per;
    };
    Frags ahead[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) ahead[i] = load(step(i));
    for (int s = 0; s < per; s += kAhead) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const Frags f = ahead[i];
            ahead[i] = load(step(s + i + kAhead));
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int a = 0; a < 2; ++a)
                    acc[a] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                        __builtin_bit_cast(bf16x8_t, f.w[a][h]),
                        __builtin_bit_cast(bf16x8_t, f.x[h]), acc[a], 0, 0, 0);
        }
    }
    if constexpr (QUARTERS) {
        if (wave > 0) {
#pragma unroll
            for (int a = 0; a < 2; ++a) part[wave - 1][a][lane] = acc[a];
        }
        __syncthreads();
        if (wave > 0) return;
    }
    if (li >= blk.rows) return;
    // rows 16a + 4*(lane/16) + v of W, row lane % 16 of the block
    int row = blk.row0 + li;
    if (g.splits == 1 && g.how_out == kRowSlot) {
        row = grouped_row(g, row, kRowSlot);
        if (row < 0) return;
    }
#pragma unroll
    for (int a = 0; a < 2; ++a) {
        f32x4_t v = acc[a];
        if constexpr (QUARTERS) {
#pragma unroll
            for (int w = 0; w < kWaves - 1; ++w) v += part[w][a][lane];
        }
        if (xoff == kNowhere) v = f32x4_t{0, 0, 0, 0};  // a padding row, whatever W holds
        const int n = a0 + 16 * a + 4 * q;
        if (n >= g.N) continue;  // N is a multiple of 8
        if (g.splits > 1)
            *reinterpret_cast<f32x4_t*>((float*)g.out + ((size_t)sp * g.R + row) * g.N + n) = v;
        else
            *reinterpret_cast<uint2*>((uint16_t*)g.out + (size_t)row * g.N + n) =
                uint2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
    }
}

}  // namespace

static bool quarters(const GroupedArgs& g) { return g.splits > 1 || g.K > kWhole; }

int grouped_stream_workgroups(const GroupedArgs& g) {
    const int blocks = g.R / kRowsB + (g.R < g.E ? g.R : g.E);
    const int rows = quarters(g) ? kRowsA : kRowsA * kWaves;
    return (g.N + rows - 1) / rows * blocks * g.splits;
}

void launch_grouped_stream_fwd(const GroupedArgs& g, hipStream_t s) {
    const int grid = grouped_stream_workgroups(g);
    if (quarters(g)) grouped_stream_kernel<true><<<grid, kWaves * 64, 0, s>>>(g);
    else grouped_stream_kernel<false><<<grid, kWaves * 64, 0, s>>>(g);
}

}  // namespace moe
