// router_bwd.hip -- the gradient of the router: from those of the routing weights
// and of the logits to the tokens, the router's weights and its bias.
//
//   dl[t,e]  = dlogits[t,e] + sum_{j: id_tj = e} w_tj (dw_tj - sum_i w_ti dw_ti)
//   dx[t,k]  = sum_j rows[t,j][k] + sum_e dl[t,e] Wr[e,k]
//   dWr[e,k] = sum_t dl[t,e] x[t,k],   dbias[e] = sum_t dl[t,e]
//
// (the weights are the softmax over the picked logits).  A first launch forms dl
// and leaves it as a sum of bf16 parts, each the rounding of what the ones before
// it left: two parts hold 16 bits of it, three all 24, and the products run on the
// bf16 matrix cores with sums in fp32.  dx, which is rounded to bf16 itself, takes
// two (off by at most 2^-16 of a term), dWr three, so nothing of dl is lost in it.
// Bound by HBM with few experts, with many by the latency of dWr's steps, whose
// workgroups are few: 4096 tokens of 4096 over 8 experts, two rows a token, 28 us
// for the products (134 MB of operands and results), 4 for dl and 4 to join dWr's
// ranges; of 7168 over 256 and eight rows 151 us (587 MB of them, 757 by the
// counters, as x is read by several tiles; dx alone 116, dWr alone 60), 7 and 6.
#include "launch.hpp"
#include "rows.hpp"
#include "small_tiles.hpp"

#include <type_traits>

namespace moe {

namespace {

constexpr int kParts = 3;       // of dl, for dWr
constexpr int kPartsDx = 2;
constexpr int kRouterCols = 2 * kSim;  // columns of k a tile

// experts of a row of a part: whole steps and tiles
__host__ __device__ inline int router_ep(int E) { return (E + kSim - 1) / kSim * kSim; }

// ---- dl -----------------------------------------------------------------------
// dl of N experts from e0 on of token t (VEC: rows of dlogits are whole vectors)
template <int N, bool VEC>
__device__ __forceinline__ void router_dl(const RouterBwdArgs& a, int t, int e0, float (&v)[N]) {
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.0f;
    if (a.dlogits) {
        const float* row = a.dlogits + (size_t)t * a.E;
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            if constexpr (VEC) {
                if (e0 + i < a.E) {
                    const f32x4_t x = *reinterpret_cast<const f32x4_t*>(row + e0 + i);
#pragma unroll
                    for (int u = 0; u < 4; ++u) v[i + u] = x[u];
                }
            } else {
#pragma unroll
                for (int u = 0; u < 4; ++u)
                    if (e0 + i + u < a.E) v[i + u] = row[e0 + i + u];
            }
        }
    }
    if (a.ids) {
        const size_t p = (size_t)t * a.topk;
        float mean = 0.0f;
        for (int j = 0; j < a.topk; ++j) mean += a.weights[p + j] * a.dweights[p + j];
        for (int j = 0; j < a.topk; ++j) {
            const int e = a.ids[p + j];
            const float g = a.weights[p + j] * (a.dweights[p + j] - mean);
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += e == e0 + i && e < a.E ? g : 0.0f;
        }
    }
}
// The next part of values, which are left with what it does not hold
__device__ __forceinline__ uint32_t next_part(float& lo, float& hi) {
    const uint32_t b = pack_bf16x2(lo, hi);
    const float x = bf16_bits_to_f32(b & 0xffffu), y = bf16_bits_to_f32(b >> 16);
    lo = __builtin_isinf(x) ? 0.0f : lo - x;  // (an infinity leaves nothing)
    hi = __builtin_isinf(y) ? 0.0f : hi - y;
    return b;
}

// L lanes a token, four experts each; parts [part][token][Ep], zeros past E.
template <int L, bool VEC>
__global__ __launch_bounds__(256) void router_dl_kernel(RouterBwdArgs a, uint16_t* __restrict__ parts) {
    const int lane = lane_id(), e0 = (lane % L) * 4, Ep = router_ep(a.E);
    const int t = ((int)blockIdx.x * 4 + (int)threadIdx.x / kWave) * (kWave / L) + lane / L;
    if (t >= a.M || e0 >= Ep) return;
    float v[4];
    router_dl<4, VEC>(a, t, e0, v);
    const size_t next = (size_t)a.M * Ep;
    uint16_t* o = parts + (size_t)t * Ep + e0;
#pragma unroll
    for (int q = 0; q < kParts; ++q)
        *reinterpret_cast<uint2*>(o + q * next) = uint2{next_part(v[0], v[1]), next_part(v[2], v[3])};
}

// ---- the products' common parts -------------------------------------------------
// A 64 x 64 piece of an operand, a thread's share of it: rows r and r + 32, chunk c
struct Piece { u16x8_t v[2]; };

__device__ __forceinline__ void put_piece(char* to, const Piece& p, bool col) {
    const int r = (int)threadIdx.x >> 3, c = (int)threadIdx.x & 7;
#pragma unroll
    for (int h = 0; h < 2; ++h)
        *reinterpret_cast<u16x8_t*>(to + (col ? sim_at<true>(r + 32 * h, c) : sim_at<false>(r + 32 * h, c))) = p.v[h];
}
// Rows of `ld` elements from `base` on, `rows` of them, columns col0..; rows of whole
// chunks through a descriptor that ends with the last row: what lies outside is
// zeros and costs no instruction.
template <Widths W>
__device__ __forceinline__ Piece get_piece(const uint16_t* base, long rows, int ld, int col0) {
    const int r = (int)threadIdx.x >> 3, c = (int)threadIdx.x & 7;
    Piece p;
    if constexpr (W == Widths::kWhole) {
        const prsrc_t src = pmake_rsrc(base, (uint32_t)(min(rows, (long)kSim) * ld * 2));
        const uint32_t col = (uint32_t)(col0 + c * 8);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint32_t at = col < (uint32_t)ld ? ((uint32_t)(r + 32 * h) * (uint32_t)ld + col) * 2 : kNowhere;
            p.v[h] = __builtin_bit_cast(u16x8_t, __builtin_amdgcn_raw_buffer_load_b128(src, at, 0, 0));
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            p.v[h] = load_chunk<W>(r + 32 * h < rows ? base + (size_t)(r + 32 * h) * ld : nullptr, col0 + c * 8, ld);
    }
    return p;
}
// The same of dl's parts, 64 tokens from t0 on and experts e0..: as the launch
// before left them, or formed here
template <int PARTS, bool IN_PLACE>
__device__ __forceinline__ void get_parts(const RouterBwdArgs& a, const uint16_t* parts, size_t t0, int e0,
                                          Piece (&d)[PARTS]) {
    const long rows = (long)a.M - (long)t0;
    if constexpr (!IN_PLACE) {
        const int Ep = router_ep(a.E);
#pragma unroll
        for (int q = 0; q < PARTS; ++q)
            d[q] = get_piece<Widths::kWhole>(parts + ((size_t)q * a.M + t0) * Ep, rows, Ep, e0);
    } else {
        const int r = (int)threadIdx.x >> 3, c = (int)threadIdx.x & 7;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            float v[8] = {};
            if (r + 32 * h < rows && e0 + c * 8 < a.E)
                router_dl<8, false>(a, (int)t0 + r + 32 * h, e0 + c * 8, v);
#pragma unroll
            for (int q = 0; q < PARTS; ++q) {
                const uint4 b = {next_part(v[0], v[1]), next_part(v[2], v[3]), next_part(v[4], v[5]),
                                 next_part(v[6], v[7])};
                d[q].v[h] = __builtin_bit_cast(u16x8_t, b);
            }
        }
    }
}
template <Widths W>
__device__ __forceinline__ void settle_piece(Piece& p, int ld, int col0) {
    if constexpr (W != Widths::kWhole) {
        if (col0 + kSim > ld) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
                p.v[h] = settle_chunk(p.v[h], col0 + ((int)threadIdx.x & 7) * 8, ld);
        }
    }
}

// ---- dx -----------------------------------------------------------------------
// 64 tokens x 128 columns a workgroup; the waves take 32 x 64.  The sums leave through
// LDS as rows of the tile, where a thread adds the tokens' rows and stores 8
// columns at a time.
template <Widths W, bool IN_PLACE>
__device__ __forceinline__ void router_dx_tile(const RouterBwdArgs& a, const uint16_t* __restrict__ parts, int tile,
                                               char* lds) {
    const int tid = (int)threadIdx.x, lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int k_tiles = (a.K + kRouterCols - 1) / kRouterCols;
    const int k0 = tile % k_tiles * kRouterCols;
    const size_t t0 = (size_t)(tile / k_tiles) * kSim;
    const int steps = (a.E + kSim - 1) / kSim;
    const long rows = (long)a.M - (long)t0;
    f32x4_t acc[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = f32x4_t{0, 0, 0, 0};
    Piece w[2], d[kPartsDx];
    auto load = [&](int s) {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            w[i] = get_piece<W>(a.w + (size_t)s * kSim * a.K, a.E - s * kSim, a.K, k0 + i * kSim);
        get_parts<kPartsDx, IN_PLACE>(a, parts, t0, s * kSim, d);
    };
    auto part = [&](int q) { return lds + (2 + q) * kSimBytes; };
    load(0);
    // four groups of 8 columns a thread, 16 tokens apart; the first rows to be added
    // are on their way while the products are formed
    constexpr bool ANY = W != Widths::kWhole;
    const int c = tid % 16, col = k0 + c * 8, n = ANY ? min(V, a.K - col) : V, first = tid / 16;
    u16x8_t row[2][4];
    auto load_rows = [&](auto at, int j) {
        constexpr int J = decltype(at)::value;
        if (col >= a.K || j >= a.rows) return;
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // (tokens past the last: the last one's, not stored)
            const size_t t = t0 + min((long)(first + i * 16), rows - 1);
            row[J][i] = ld_bf16_bits<ANY, true>(a.dx_rows + (t * a.rows + j) * a.K + col, n, a.K >= V);
        }
    };
    const std::integral_constant<int, 0> even;
    const std::integral_constant<int, 1> odd;
    load_rows(even, 0);
    load_rows(odd, 1);
    for (int s = 0; s < steps; ++s) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            settle_piece<W>(w[i], a.K, k0 + i * kSim);
            put_piece(lds + i * kSimBytes, w[i], true);
        }
#pragma unroll
        for (int q = 0; q < kPartsDx; ++q) put_piece(part(q), d[q], false);
        __syncthreads();
        if (s + 1 < steps) load(s + 1);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            if (s * kSim + ks * 32 >= a.E) break;
            bf16x8_t fa[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) fa[i] = sim_frag<true>(lds + (wave & 1) * kSimBytes, 16 * i, ks, lane);
#pragma unroll
            for (int q = 0; q < kPartsDx; ++q) {
                bf16x8_t fb[2];
#pragma unroll
                for (int j = 0; j < 2; ++j) fb[j] = sim_frag<false>(part(q), (wave >> 1) * 32 + 16 * j, ks, lane);
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
            }
        }
        __syncthreads();
    }
    // chunks of four columns, permuted by the token
    auto at = [](int token, int chunk) { return token * (kRouterCols * 4) + ((chunk ^ (token & 15)) << 4); };
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j)
            *reinterpret_cast<f32x4_t*>(lds + at((wave >> 1) * 32 + 16 * j + (lane & 15),
                                                 (wave & 1) * 16 + 4 * i + (lane >> 4))) = acc[i][j];
    __syncthreads();
    if (col >= a.K) return;
    float f[4][V];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const f32x4_t v = *reinterpret_cast<const f32x4_t*>(lds + at(first + i * 16, 2 * c + u));
#pragma unroll
            for (int x = 0; x < 4; ++x) f[i][4 * u + x] = v[x];
        }
    auto add_rows = [&](auto at, int j) {
        constexpr int J = decltype(at)::value;
        if (j >= a.rows) return;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int u = 0; u < V; ++u) f[i][u] += bf16_bits_to_f32(row[J][i][u]);
        load_rows(at, j + 2);
    };
    for (int j = 0; j < a.rows; j += 2) {
        add_rows(even, j);
        add_rows(odd, j + 1);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (first + i * 16 < rows) st_bf16<ANY, true>(a.dx + (t0 + first + i * 16) * a.K + col, n, f[i]);
}

// ---- dWr ----------------------------------------------------------------------
// 64 experts x 128 columns a workgroup over a range of the tokens; the waves take 32
// x 64.  One range writes the results, more leave [range][E][ld] with the bias' sums
// behind a row.
__host__ __device__ inline int router_ld(int K) { return (K + 3) / 4 * 4 + 4; }

template <Widths W, bool IN_PLACE>
__device__ __forceinline__ void router_dw_tile(const RouterBwdArgs& a, const uint16_t* __restrict__ parts, int splits,
                                               float* __restrict__ sums, int tile, char* lds) {
    const int tid = (int)threadIdx.x, lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int k_tiles = (a.K + kRouterCols - 1) / kRouterCols, e_tiles = (a.E + kSim - 1) / kSim;
    int b = tile;
    const int e0 = b % e_tiles * kSim;
    b /= e_tiles;
    const int k0 = b % k_tiles * kRouterCols, sp = b / k_tiles;
    const int all = (a.M + kSim - 1) / kSim, per = (all + splits - 1) / splits;
    const int first = min(sp * per, all), steps = min(per, all - first);
    f32x4_t acc[4][2];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[i][j] = f32x4_t{0, 0, 0, 0};
    // the bias: the same product with a column of ones, 16 experts a wave
    const bool with_bias = a.dbias && k0 == 0;
    f32x4_t bias = {0, 0, 0, 0};
    bf16x8_t ones;
#pragma unroll
    for (int i = 0; i < 8; ++i) ones[i] = 0x3f80;
    Piece x[2], d[kParts];
    auto load = [&](int s) {
        const size_t t0 = (size_t)(first + s) * kSim;
        const long rows = (long)a.M - (long)t0;
#pragma unroll
        for (int i = 0; i < 2; ++i) x[i] = get_piece<W>(a.x + t0 * a.K, rows, a.K, k0 + i * kSim);
        get_parts<kParts, IN_PLACE>(a, parts, t0, e0, d);
    };
    auto part = [&](int q) { return lds + (2 + q) * kSimBytes; };
    if (steps > 0) load(0);
    for (int s = 0; s < steps; ++s) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            settle_piece<W>(x[i], a.K, k0 + i * kSim);
            put_piece(lds + i * kSimBytes, x[i], true);
        }
#pragma unroll
        for (int q = 0; q < kParts; ++q) put_piece(part(q), d[q], true);
        __syncthreads();
        if (s + 1 < steps) load(s + 1);
        const int row0 = (wave >> 1) * 32;  // experts of the tile that the wave takes
        if (e0 + row0 < a.E) {
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
                bf16x8_t fa[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) fa[i] = sim_frag<true>(lds + (wave & 1) * kSimBytes, 16 * i, ks, lane);
#pragma unroll
                for (int q = 0; q < kParts; ++q) {
                    bf16x8_t fb[2];
#pragma unroll
                    for (int j = 0; j < 2; ++j) fb[j] = sim_frag<true>(part(q), row0 + 16 * j, ks, lane);
                    if (with_bias)
                        bias = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, wave & 1 ? fb[1] : fb[0], bias, 0, 0, 0);
#pragma unroll
                    for (int i = 0; i < 4; ++i)
#pragma unroll
                        for (int j = 0; j < 2; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fa[i], fb[j], acc[i][j], 0, 0, 0);
                }
            }
        }
        __syncthreads();
    }
    const int ld = splits > 1 ? router_ld(a.K) : a.K;
    float* out = splits > 1 ? sums + (size_t)sp * a.E * ld : a.dw;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int e = e0 + (wave >> 1) * 32 + 16 * j + (lane & 15);
        if (e >= a.E) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int col = k0 + (wave & 1) * kSim + 16 * i + 4 * (lane >> 4);
            float* o = out + (size_t)e * ld + col;
            if (col + 4 <= a.K) {
                *reinterpret_cast<f32x4_any_t*>(o) = acc[i][j];
            } else {
#pragma unroll
                for (int u = 0; u < 3; ++u)
                    if (col + u < a.K) o[u] = acc[i][j][u];
            }
        }
    }
    if (with_bias && lane < 16) {  // (every row of the product is the sum)
        const int e = e0 + (wave >> 1) * 32 + (wave & 1) * 16 + lane;
        if (e < a.E) {
            if (splits > 1) out[(size_t)e * ld + ld - 4] = bias[0];
            else a.dbias[e] = bias[0];
        }
    }
}

// Both products in one launch: dWr's tiles, which take long and wait for their steps,
// first, and dx's, which are bound by HBM, beside and behind them (us a call, so / dx's
// first: 4096 x 7168 over 256 157/182, 8192 x 4096 over 64 84/90, 4096 x 4096 over 8
// 34.2/34.5).  Three workgroups a CU leave 168 registers: the variants that form dl in
// place at widths that are no multiples of 8 spill 3 of them, below 8 columns 17 (calls
// of up to 128 tokens, which wait for the host).
template <Widths W, bool IN_PLACE>
__global__ __launch_bounds__(256, 3) void router_products_kernel(RouterBwdArgs a, const uint16_t* __restrict__ parts,
                                                                 int splits, float* __restrict__ sums, int dw_tiles) {
    __shared__ __attribute__((aligned(16))) char lds[(2 + kParts) * kSimBytes];
    static_assert((2 + kParts) * kSimBytes >= kSim * kRouterCols * 4, "dx's tile in fp32 takes the pieces' place");
    const int b = (int)blockIdx.x;
    // (the hardware deals workgroup g to XCD g % 8: an XCD takes neighbouring tiles
    // of dWr, whose tokens its L2 then holds for all of a column's experts)
    const int per_xcd = (dw_tiles + 7) / 8;
    if (b < 8 * per_xcd) {
        const int tile = b % 8 * per_xcd + b / 8;
        if (tile < dw_tiles) router_dw_tile<W, IN_PLACE>(a, parts, splits, sums, tile, lds);
    } else {
        router_dx_tile<W, IN_PLACE>(a, parts, b - 8 * per_xcd, lds);
    }
}

// the ranges' sums in order, a thread per four values; the last four of a row: the bias
__global__ __launch_bounds__(256) void router_join_kernel(RouterBwdArgs a, int splits,
                                                          const float* __restrict__ sums) {
    const int ld = router_ld(a.K);
    const uint32_t at = blockIdx.x * 256u + threadIdx.x;
    const int e = (int)(at / (uint32_t)(ld / 4)), col = (int)(at % (uint32_t)(ld / 4)) * 4;
    if (e >= a.E) return;
    const bool bias = col == ld - 4;
    if (bias && !a.dbias) return;
    const float* p = sums + (size_t)e * ld + col;
    const size_t next = (size_t)a.E * ld;
    f32x4_t v = *reinterpret_cast<const f32x4_t*>(p);
#pragma unroll 4
    for (int s = 1; s < splits; ++s) v += *reinterpret_cast<const f32x4_t*>(p + s * next);
    if (bias) {
        a.dbias[e] = v[0];
        return;
    }
    float* o = a.dw + (size_t)e * a.K + col;
    if (col + 4 <= a.K) {
        *reinterpret_cast<f32x4_any_t*>(o) = v;
    } else {
#pragma unroll
        for (int u = 0; u < 3; ++u)
            if (col + u < a.K) o[u] = v[u];
    }
}

struct RouterPlan {
    bool in_place;  // no launch for dl
    int splits;     // ranges the tokens are cut into, for dWr
    int k_tiles, dw_tiles, dx_tiles;
};
RouterPlan router_plan(int M, int K, int E) {
    RouterPlan p;
    // us a call, formed in place / by a launch of its own: 64 tokens of 4096 over 8
    // experts 13.0/17, 128 of 4096 over 8 13.4/17.1, of 1024 over 64 16.1/16.8, 190 of
    // 4096 over 64 22.6/16.8, 64 of 1024 over 128 17.1/16.7
    p.in_place = M <= 2 * kSim && E <= kSim;
    p.k_tiles = (K + kRouterCols - 1) / kRouterCols;
    const int steps = (M + kSim - 1) / kSim;
    const long tiles = (long)((E + kSim - 1) / kSim) * p.k_tiles;
    // Ranges of the tokens up to two workgroups of dWr a CU, while one has four steps
    // and the whole 12: ranges are a third launch, which costs a stream of calls 2-4 us
    // on the host.  us a call, whole / in two (the same in a captured graph): 512 tokens
    // of 4096 over 8 17.2/20.9 (14.2/12.1), 704 18.3/20.8 (18.2/14.5), 768 19.3/20.9
    // (19.4/15.0), 1024 24.6/20.9 (24.8/18.6); of 1024 over 64 512 18.2/20.4 (14.8/12.9),
    // 768 19.6/20.4 (19.5/14.7), 1024 24.5/19.7 (24.3/17.4).  So from 8 to 11 steps a
    // graph pays 2-4 us for what a stream saves, at 12 and 13 the stream one for what
    // the graph saves; and where the tiles are many, 12 steps are few: 768 of 7168 over
    // 256 39.4/43.0 (39.6/43.2).  Up to four workgroups a CU: 4096 of these 172 against 163.
    p.splits = 1;
    while (steps >= 12 && p.splits < 64 && tiles * p.splits * 2 <= 512 && steps / (p.splits * 2) >= 4) p.splits *= 2;
    p.dw_tiles = (int)(tiles * p.splits);
    p.dx_tiles = (int)((long)steps * p.k_tiles);
    return p;
}

// tokens of a workgroup of dl's launch: 16 lanes a token up to 64 experts, then 32, 64
int router_dl_tokens(int E) { return E <= 64 ? 16 : E <= 128 ? 8 : 4; }

size_t parts_bytes(int M, int E) { return ((size_t)kParts * M * router_ep(E) * 2 + 255) / 256 * 256; }

}  // namespace

long router_bwd_workgroups(int M, int K, int E) {
    const RouterPlan p = router_plan(M, K, E);
    const long products = (long)p.k_tiles * ((M + kSim - 1) / kSim + p.splits * ((E + kSim - 1) / kSim)) + 7;
    const int tokens = router_dl_tokens(E);
    const long dl = p.in_place ? 0 : ((long)M + tokens - 1) / tokens;
    return products > dl ? products : dl;
}

size_t router_bwd_workspace(int M, int K, int E) {
    const RouterPlan plan = router_plan(M, K, E);
    const int splits = plan.splits;
    return plan.in_place ? 0 : parts_bytes(M, E) + (splits > 1 ? (size_t)splits * E * router_ld(K) * 4 : 0);
}

void launch_router_bwd(const RouterBwdArgs& a, void* workspace, hipStream_t s) {
    uint16_t* parts = (uint16_t*)workspace;
    float* sums = (float*)((char*)workspace + parts_bytes(a.M, a.E));
    const RouterPlan plan = router_plan(a.M, a.K, a.E);
    if (a.M > 0 && !plan.in_place) {
        auto dl = [&](auto lanes) {
            constexpr int L = decltype(lanes)::value;
            const int tokens = router_dl_tokens(a.E), grid = (a.M + tokens - 1) / tokens;
            if (a.E % 4 == 0) router_dl_kernel<L, true><<<grid, 256, 0, s>>>(a, parts);
            else router_dl_kernel<L, false><<<grid, 256, 0, s>>>(a, parts);
        };
        if (a.E <= 64) dl(std::integral_constant<int, 16>{});
        else if (a.E <= 128) dl(std::integral_constant<int, 32>{});
        else dl(std::integral_constant<int, 64>{});
    }
    const int grid = (plan.dw_tiles + 7) / 8 * 8 + plan.dx_tiles;
    auto products = [&](auto width) {
        constexpr Widths W = decltype(width)::value;
        if (plan.in_place)
            router_products_kernel<W, true><<<grid, 256, 0, s>>>(a, parts, plan.splits, sums, plan.dw_tiles);
        else
            router_products_kernel<W, false><<<grid, 256, 0, s>>>(a, parts, plan.splits, sums, plan.dw_tiles);
    };
    if (a.K % 8 == 0) products(std::integral_constant<Widths, Widths::kWhole>{});
    else if (a.K >= 8) products(std::integral_constant<Widths, Widths::kLong>{});
    else products(std::integral_constant<Widths, Widths::kAny>{});
    if (plan.splits > 1) {
        const long threads = (long)a.E * (router_ld(a.K) / 4);
        router_join_kernel<<<(int)((threads + 255) / 256), 256, 0, s>>>(a, plan.splits, sums);
    }
}

}  // namespace moe
