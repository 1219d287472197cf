// ckpt.hip -- activations kept in 8 bits for the backward pass (the format:
// ckpt.hpp): rows of bf16 to codes and back, and the gated activation that
// keeps its input on the way forward and reads it on the way back.
//
//   a[i,n]  = w[p] silu(g[i,n]) u[i,n];   g^, u^ = what is kept of g, u
//   dg[i,n] = da w u^ s(g^) (1 + g^ (1 - s(g^))),   du[i,n] = da w silu(g^)
//   dw[p]   = sum_n da[i,n] silu(g^[i,n]) u^[i,n],  a^[i,n] = w[p] silu(g^) u^
//
// All are bound by HBM: every value is read and written once, 16 bytes of bf16 or
// 8 of codes a lane; a quad of lanes holds a block.  Arithmetic is fp32.
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
__device__ __forceinline__ CkptPlace ckpt_place(int R, int W) {
    const uint32_t per_row = (uint32_t)ckpt_blocks(W) * kCkptLanes;
    const uint32_t at = blockIdx.x * 256u + threadIdx.x;  // a launch has at most 2^32 threads
    const uint32_t i = at / per_row;
    CkptPlace p;
    p.i = (int)i;
    p.block = (int)((at - i * per_row) / kCkptLanes);
    p.col = (int)(at - i * per_row) * V;
    p.n = i < (uint32_t)R ? min(V, W - p.col) : 0;
    return p;
}

template <bool ANY>
__global__ __launch_bounds__(256) void ckpt_rows_kernel(const uint16_t* __restrict__ x, int R, int W,
                                                        int8_t* __restrict__ codes,
                                                        uint8_t* __restrict__ scales) {
    const CkptPlace p = ckpt_place(R, W);
    const size_t at = (size_t)p.i * W + p.col;
    const u16x8_t v = ld_bf16_bits<ANY, true>(x + at, p.n);
    const uint32_t X = ckpt_quad_power(v);
    if (p.n <= 0) return;
    st_codes<ANY>(codes + at, p.n, ckpt_codes(v, X));
    if (threadIdx.x % kCkptLanes == 0) scales[(size_t)p.i * ckpt_blocks(W) + p.block] = (uint8_t)X;
}

template <bool ANY>
__global__ __launch_bounds__(256) void ckpt_restore_kernel(const int8_t* __restrict__ codes,
                                                           const uint8_t* __restrict__ scales, int R,
                                                           int W, uint16_t* __restrict__ x) {
    const CkptPlace p = ckpt_place(R, W);
    if (p.n <= 0) return;
    const size_t at = (size_t)p.i * W + p.col;
    float f[V];
    ckpt_values(ld_codes<ANY>(codes + at, p.n), scales[(size_t)p.i * ckpt_blocks(W) + p.block], f);
    st_bf16<ANY>(x + at, p.n, f);
}

template <bool ANY>
__global__ __launch_bounds__(256) void silu_mul_ckpt_kernel(GatedCkptArgs a) {
    const CkptPlace t = ckpt_place(a.R, a.N);
    const int p = t.n > 0 ? gated_slot(a, t.i) : -2;  // the same for a quad but for lanes without columns
    const int nb = ckpt_blocks(a.N);
    const size_t at = (size_t)t.i * 2 * a.N + t.col;
    const u16x8_t g = ld_bf16_bits<ANY, true>(a.g + at, p >= 0 ? t.n : 0);
    const u16x8_t u = ld_bf16_bits<ANY, true>(a.g + at + a.N, p >= 0 ? t.n : 0);
    const uint32_t Xg = ckpt_quad_power(g), Xu = ckpt_quad_power(u);
    if (p == -2) return;
    float y[V] = {};
    if (p >= 0) {
        const float w = a.weights ? a.weights[p] : 1.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) y[v] = w * silu(bf16_bits_to_f32(g[v])) * bf16_bits_to_f32(u[v]);
    }
    st_bf16<ANY, true>(a.out + (size_t)t.i * a.N + t.col, t.n, y);
    st_codes<ANY, true>(a.codes_out + at, t.n, ckpt_codes(g, Xg));
    st_codes<ANY, true>(a.codes_out + at + a.N, t.n, ckpt_codes(u, Xu));
    if (threadIdx.x % kCkptLanes == 0) {
        uint8_t* s = a.scales_out + (size_t)t.i * 2 * nb + t.block;
        s[0] = (uint8_t)Xg;
        s[nb] = (uint8_t)Xu;
    }
}

// a workgroup per row
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
    float dot = 0.0f;
    for (int col = (int)threadIdx.x * V; col < a.N; col += TH * V) {
        const int n = ANY ? min(V, a.N - col) : V;
        float dg[V] = {}, du[V] = {}, act[V] = {};
        if (p >= 0) {
            float z[V], u[V], da[V];
            const u32x2_t cz = ld_codes<ANY, true>(g + col, n), cu = ld_codes<ANY, true>(g + a.N + col, n);
            const uint32_t Xz = sc[col / kCkptBlock], Xu = sc[nb + col / kCkptBlock];
            ld_bf16<ANY, true>(d + col, n, da);
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
        if (again) st_bf16<ANY, true>(again + col, n, act);
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

int ckpt_grid(int R, int W) {
    return (int)(((long)R * ckpt_blocks(W) * kCkptLanes + 255) / 256);
}

}  // namespace

void launch_ckpt_rows(const uint16_t* x, int R, int W, int8_t* codes, uint8_t* scales, hipStream_t s) {
    const int grid = ckpt_grid(R, W);
    if (W % V == 0) ckpt_rows_kernel<false><<<grid, 256, 0, s>>>(x, R, W, codes, scales);
    else ckpt_rows_kernel<true><<<grid, 256, 0, s>>>(x, R, W, codes, scales);
}

void launch_ckpt_restore(const int8_t* codes, const uint8_t* scales, int R, int W, uint16_t* x,
                         hipStream_t s) {
    const int grid = ckpt_grid(R, W);
    if (W % V == 0) ckpt_restore_kernel<false><<<grid, 256, 0, s>>>(codes, scales, R, W, x);
    else ckpt_restore_kernel<true><<<grid, 256, 0, s>>>(codes, scales, R, W, x);
}

void launch_silu_mul_ckpt(const GatedCkptArgs& a, hipStream_t s) {
    const int grid = ckpt_grid(a.R, a.N);
    if (a.N % V == 0) silu_mul_ckpt_kernel<false><<<grid, 256, 0, s>>>(a);
    else silu_mul_ckpt_kernel<true><<<grid, 256, 0, s>>>(a);
}

void launch_silu_mul_bwd_ckpt(const GatedCkptArgs& a, hipStream_t s) {
    auto run = [&](auto any) {
        constexpr bool ANY = decltype(any)::value;
        if (a.N <= kWave * V) silu_mul_bwd_ckpt_kernel<kWave, ANY><<<a.R, kWave, 0, s>>>(a);
        else silu_mul_bwd_ckpt_kernel<256, ANY><<<a.R, 256, 0, s>>>(a);
    };
    if (a.N % V == 0) run(std::false_type{});
    else run(std::true_type{});
}

}  // namespace moe
