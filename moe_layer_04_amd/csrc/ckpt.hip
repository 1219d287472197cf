// ckpt.hip -- activations kept in 8 bits for the backward pass (the format:
// ckpt.hpp): rows of bf16 to codes and back, and the gated activation that
// keeps its input on the way forward and reads it on the way back.
//
//   a[i,n]  = w[p] silu(g[i,n]) u[i,n];   g^, u^ = what is kept of g, u
//   dg[i,n] = da w u^ s(g^) (1 + g^ (1 - s(g^))),   du[i,n] = da w silu(g^)
//   dw[p]   = sum_n da[i,n] silu(g^[i,n]) u^[i,n],  a^[i,n] = w[p] silu(g^) u^
//
// All are bound by HBM: every value is read and written once, 16 bytes of bf16 or
// 8 of codes a lane; a quad of lanes holds a block.  Arithmetic is fp32.  8192 x
// 7168: to codes 31.5 us (5.6 TB/s), back 26.3 (6.8); the activation of 8192 x 14336
// forward 158-167 us (5.7-6.0 TB/s), backward 176-181 (6.5-6.7); rows that are no
// multiple of 8 long 4.2-5.4 TB/s.  Codes stay in the L2 (past it the forward took
// 164 us against 157, ckpt_rows 34.8 against 32.9).
#include "ckpt.hpp"
#include "gated.hpp"

#include <type_traits>

namespace moe {

namespace {

// Where a thread works: a quad a block of a row's 32 columns.  Lanes without
// columns (n <= 0) stay for the quad's exchange.
struct CkptPlace {
    int i, block, col, n;
};
__device__ __forceinline__ CkptPlace ckpt_place(int R, int W, uint32_t group = blockIdx.x) {
    const uint32_t per_row = (uint32_t)ckpt_blocks(W) * kCkptLanes;
    const uint32_t at = group * 256u + threadIdx.x;  // below 2^32 in all
    const uint32_t i = at / per_row;
    CkptPlace p;
    p.i = (int)i;
    p.block = (int)((at - i * per_row) / kCkptLanes);
    p.col = (int)(at - i * per_row) * V;
    p.n = i < (uint32_t)R ? min(V, W - p.col) : 0;
    return p;
}

// U groups of 8 columns a thread, 256 apart
template <bool ANY, int U>
__global__ __launch_bounds__(256) void ckpt_rows_kernel(const uint16_t* __restrict__ x, int R, int W,
                                                        int8_t* __restrict__ codes,
                                                        uint8_t* __restrict__ scales) {
    CkptPlace p[U];
    u16x8_t v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        p[u] = ckpt_place(R, W, blockIdx.x * U + u);
        v[u] = ld_bf16_bits<ANY, true>(x + (size_t)p[u].i * W + p[u].col, p[u].n, W >= V);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t X = ckpt_quad_power(v[u]);
        if (p[u].n <= 0) continue;
        st_codes<ANY>(codes + (size_t)p[u].i * W + p[u].col, p[u].n, ckpt_codes(v[u], X));
        if (threadIdx.x % kCkptLanes == 0) scales[(size_t)p[u].i * ckpt_blocks(W) + p[u].block] = (uint8_t)X;
    }
}

template <bool ANY, int U>
__global__ __launch_bounds__(256) void ckpt_restore_kernel(const int8_t* __restrict__ codes,
                                                           const uint8_t* __restrict__ scales, int R,
                                                           int W, uint16_t* __restrict__ x) {
    CkptPlace p[U];
    u32x2_t w[U];
    uint32_t X[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        p[u] = ckpt_place(R, W, blockIdx.x * U + u);
        if (p[u].n <= 0) continue;
        w[u] = ld_codes<ANY>(codes + (size_t)p[u].i * W + p[u].col, p[u].n, W >= V);
        X[u] = scales[(size_t)p[u].i * ckpt_blocks(W) + p[u].block];
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (p[u].n <= 0) continue;
        float f[V];
        ckpt_values(w[u], X[u], f);
        st_bf16<ANY>(x + (size_t)p[u].i * W + p[u].col, p[u].n, f);
    }
}

template <bool ANY, int U>
__global__ __launch_bounds__(256) void silu_mul_ckpt_kernel(GatedCkptArgs a) {
    CkptPlace t[U];
    int p[U];
    u16x8_t g[U], u[U];
    const int nb = ckpt_blocks(a.N);
#pragma unroll
    for (int k = 0; k < U; ++k) {
        t[k] = ckpt_place(a.R, a.N, blockIdx.x * U + k);
        // (the same for a quad but for lanes without columns)
        p[k] = t[k].n > 0 ? gated_slot(a, t[k].i) : -2;
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const uint16_t* row = a.g + (size_t)t[k].i * 2 * a.N + t[k].col;
        g[k] = ld_bf16_bits<ANY, true>(row, p[k] >= 0 ? t[k].n : 0, a.N >= V);
        u[k] = ld_bf16_bits<ANY, true>(row + a.N, p[k] >= 0 ? t[k].n : 0, a.N >= V);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const uint32_t Xg = ckpt_quad_power(g[k]), Xu = ckpt_quad_power(u[k]);
        if (p[k] == -2) continue;
        const size_t at = (size_t)t[k].i * 2 * a.N + t[k].col;
        float y[V] = {};
        if (p[k] >= 0) {
            const float w = a.weights ? a.weights[p[k]] : 1.0f;
#pragma unroll
            for (int v = 0; v < V; ++v) y[v] = w * silu(bf16_bits_to_f32(g[k][v])) * bf16_bits_to_f32(u[k][v]);
        }
        st_bf16<ANY, true>(a.out + (size_t)t[k].i * a.N + t[k].col, t[k].n, y);
        st_codes<ANY>(a.codes_out + at, t[k].n, ckpt_codes(g[k], Xg));
        st_codes<ANY>(a.codes_out + at + a.N, t[k].n, ckpt_codes(u[k], Xu));
        if (threadIdx.x % kCkptLanes == 0) {
            uint8_t* s = a.scales_out + (size_t)t[k].i * 2 * nb + t[k].block;
            s[0] = (uint8_t)Xg;
            s[nb] = (uint8_t)Xu;
        }
    }
}

// A workgroup per row, of as many threads as the row has groups of 8 columns, rounded
// down to a power of two: fewer leave loads too far apart (us of 64 / 128 / 256 / 512
// / 1024 threads: 8192 x 14336 207 / 201 / 190 / 180 / 171, 16384 x 7168 195 / 187 / 178
// / 170 / 179, 32768 x 2048 102 / 100 / 96 / 107 / 167), and more idle.  The forward's
// output again stays in the L2 (8192 x 14336: 171 us, 199 past it).
template <int TH, bool ANY>
__global__ __launch_bounds__(TH) void silu_mul_bwd_ckpt_kernel(GatedCkptArgs a) {
    __shared__ float part[TH / kWave];
    const int i = (int)blockIdx.x;
    const int p = gated_slot(a, i);
    if (p == -2) return;
    const float w = p >= 0 && a.weights ? a.weights[p] : 1.0f;
    const int nb = ckpt_blocks(a.N);
    const int8_t* g = a.codes + (size_t)i * 2 * a.N;
    const uint8_t* sc = a.scales + (size_t)i * 2 * nb;
    const uint16_t* d = a.da + (size_t)i * a.N;
    uint16_t* o = a.out + (size_t)i * 2 * a.N;
    uint16_t* again = a.again ? a.again + (size_t)i * a.N : nullptr;
    const bool wide = a.N >= V;
    float dot = 0.0f;
    for (int col = (int)threadIdx.x * V; col < a.N; col += TH * V) {
        const int n = ANY ? min(V, a.N - col) : V;
        float dg[V] = {}, du[V] = {}, act[V] = {};
        if (p >= 0) {
            float z[V], u[V], da[V];
            const u32x2_t cz = ld_codes<ANY, true>(g + col, n, wide), cu = ld_codes<ANY, true>(g + a.N + col, n, wide);
            const uint32_t Xz = sc[col / kCkptBlock], Xu = sc[nb + col / kCkptBlock];
            ld_bf16<ANY, true>(d + col, n, wide, da);
            ckpt_values(cz, Xz, z);
            ckpt_values(cu, Xu, u);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-z[v]));
                const float h = z[v] * s;
                act[v] = w * h * u[v];
                // (columns past the row's end would add the zeros of da to a NaN block's values)
                dot += ANY && v >= n ? 0.0f : da[v] * h * u[v];
                dg[v] = da[v] * w * u[v] * (s + h * (1.0f - s));
                du[v] = da[v] * w * h;
            }
        }
        st_bf16<ANY, true>(o + col, n, dg);
        st_bf16<ANY, true>(o + a.N + col, n, du);
        if (again) st_bf16<ANY>(again + col, n, act);
    }
    if (!a.dweights || p < 0) return;  // the same for the whole workgroup
    dot = wave_sum_f32(dot);
    if constexpr (TH > kWave) {
        if (lane_id() == 0) part[threadIdx.x / kWave] = dot;
        __syncthreads();
        dot = part[0];
#pragma unroll
        for (int k = 1; k < TH / kWave; ++k) dot += part[k];
    }
    if (threadIdx.x == 0) a.dweights[p] = dot;
}

constexpr int kU = 2;  // groups of 8 columns a thread (8192 x 7168: to codes 31.6 us, 33.4 with one)
int ckpt_grid(int R, int W) {
    return (int)(((long)R * ckpt_blocks(W) * kCkptLanes + 255) / 256);
}

}  // namespace

void launch_ckpt_rows(const uint16_t* x, int R, int W, int8_t* codes, uint8_t* scales, hipStream_t s) {
    const int grid = (ckpt_grid(R, W) + kU - 1) / kU;
    if (W % V == 0) ckpt_rows_kernel<false, kU><<<grid, 256, 0, s>>>(x, R, W, codes, scales);
    else ckpt_rows_kernel<true, kU><<<grid, 256, 0, s>>>(x, R, W, codes, scales);
}

void launch_ckpt_restore(const int8_t* codes, const uint8_t* scales, int R, int W, uint16_t* x,
                         hipStream_t s) {
    const int grid = (ckpt_grid(R, W) + kU - 1) / kU;
    if (W % V == 0) ckpt_restore_kernel<false, kU><<<grid, 256, 0, s>>>(codes, scales, R, W, x);
    else ckpt_restore_kernel<true, kU><<<grid, 256, 0, s>>>(codes, scales, R, W, x);
}

void launch_silu_mul_ckpt(const GatedCkptArgs& a, hipStream_t s) {
    const int grid = (ckpt_grid(a.R, a.N) + kU - 1) / kU;
    if (a.N % V == 0) silu_mul_ckpt_kernel<false, kU><<<grid, 256, 0, s>>>(a);
    else silu_mul_ckpt_kernel<true, kU><<<grid, 256, 0, s>>>(a);
}

void launch_silu_mul_bwd_ckpt(const GatedCkptArgs& a, hipStream_t s) {
    auto run = [&](auto threads) {
        constexpr int TH = decltype(threads)::value;
        if (a.N % V == 0) silu_mul_bwd_ckpt_kernel<TH, false><<<a.R, TH, 0, s>>>(a);
        else silu_mul_bwd_ckpt_kernel<TH, true><<<a.R, TH, 0, s>>>(a);
    };
    const int vectors = a.N / V;
    if (vectors < 128) run(std::integral_constant<int, 64>{});
    else if (vectors < 256) run(std::integral_constant<int, 128>{});
    else if (vectors < 512) run(std::integral_constant<int, 256>{});
    else if (vectors < 1024) run(std::integral_constant<int, 512>{});
    else run(std::integral_constant<int, 1024>{});
}

}  // namespace moe
