// gated_act.hip -- the gated activation between an expert's two products,
// with the routing weight of the row, and its gradients:
//
//   a[i,n]  = w[p] silu(g[i,n]) u[i,n],   silu(z) = z s(z), s(z) = 1/(1+e^-z)
//   dg[i,n] = da w u s(g) (1 + g (1 - s(g)))
//   du[i,n] = da w silu(g)
//   dw[p]   = sum_n da[i,n] silu(g[i,n]) u[i,n]
//
// p = sorted[i] is the row's slot.  Rows hold the gate half, then the up
// half.  Both passes are bound by HBM: every value is read and written once, 16
// bytes a lane; arithmetic and the row's dot product are fp32.
// 8192 x 14336: backward 211 us (5.6 TB/s), forward 106 us (6.6 TB/s), by loads and
// stores that keep nothing in the L2 (219 and 117 us by ordinary ones); 16 x
// 14336: forward 2.7 us, a launch.
#include "gated.hpp"
#include "rows.hpp"

#include <type_traits>

namespace moe {

namespace {

// a thread per 8 columns, rows one after the other
template <bool ANY>
__global__ __launch_bounds__(256) void silu_mul_kernel(GatedArgs a) {
    const uint32_t per_row = ((uint32_t)a.N + V - 1) / V;
    const uint32_t at = blockIdx.x * 256u + threadIdx.x;  // a launch has at most 2^32 threads
    const uint32_t i = at / per_row;
    if (i >= (uint32_t)a.R) return;
    const int col = (int)(at - i * per_row) * V, n = ANY ? min(V, a.N - col) : V;
    const int p = gated_slot(a, (int)i);
    if (p == -2) return;
    const uint16_t* g = a.g + (size_t)i * 2 * a.N + col;
    float y[V] = {};
    if (p >= 0) {
        const float w = a.weights ? a.weights[p] : 1.0f;
        float z[V], u[V];
        ld_bf16<ANY, true>(g, n, z);
        ld_bf16<ANY, true>(g + a.N, n, u);
#pragma unroll
        for (int v = 0; v < V; ++v) y[v] = w * silu(z[v]) * u[v];
    }
    st_bf16<ANY, true>(a.out + (size_t)i * a.N + col, n, y);
}

// a workgroup per row
template <int TH, bool ANY>
__global__ __launch_bounds__(TH) void silu_mul_bwd_kernel(GatedArgs a) {
    __shared__ float part[TH / kWave];
    const int i = (int)blockIdx.x;
    const int p = gated_slot(a, i);
    if (p == -2) return;
    const float w = p >= 0 && a.weights ? a.weights[p] : 1.0f;
    const uint16_t* g = a.g + (size_t)i * 2 * a.N;
    const uint16_t* d = a.da + (size_t)i * a.N;
    uint16_t* o = a.out + (size_t)i * 2 * a.N;
    float dot = 0.0f;
    for (int col = (int)threadIdx.x * V; col < a.N; col += TH * V) {
        const int n = ANY ? min(V, a.N - col) : V;
        float dg[V] = {}, du[V] = {};
        if (p >= 0) {
            float z[V], u[V], da[V];
            ld_bf16<ANY, true>(g + col, n, z);
            ld_bf16<ANY, true>(g + a.N + col, n, u);
            ld_bf16<ANY, true>(d + col, n, da);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-z[v]));
                const float act = z[v] * s;
                dot += da[v] * act * u[v];
                dg[v] = da[v] * w * u[v] * (s + act * (1.0f - s));
                du[v] = da[v] * w * act;
            }
        }
        st_bf16<ANY, true>(o + col, n, dg);
        st_bf16<ANY, true>(o + a.N + col, n, du);
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

}  // namespace

void launch_silu_mul(const GatedArgs& a, hipStream_t s) {
    const long threads = (long)a.R * ((a.N + V - 1) / V);
    const int grid = (int)((threads + 255) / 256);
    if (a.N % V == 0) silu_mul_kernel<false><<<grid, 256, 0, s>>>(a);
    else silu_mul_kernel<true><<<grid, 256, 0, s>>>(a);
}

void launch_silu_mul_bwd(const GatedArgs& a, hipStream_t s) {
    auto run = [&](auto any) {
        constexpr bool ANY = decltype(any)::value;
        if (a.N <= kWave * V) silu_mul_bwd_kernel<kWave, ANY><<<a.R, kWave, 0, s>>>(a);
        else silu_mul_bwd_kernel<256, ANY><<<a.R, 256, 0, s>>>(a);
    };
    if (a.N % V == 0) run(std::false_type{});
    else run(std::true_type{});
}

}  // namespace moe
