// gated_act.hip -- the gated activation between an expert's two products,
// with the routing weight of the row, and its gradients:
//
//   a[i,n]  = w[p] silu(g[i,n]) u[i,n],   silu(z) = z s(z), s(z) = 1/(1+e^-z)
//   dg[i,n] = da w u s(g) (1 + g (1 - s(g)))
//   du[i,n] = da w silu(g)
//   dw[p]   = sum_n da[i,n] silu(g[i,n]) u[i,n]
//
// p = sorted[i] is the row's slot.  Rows hold the gate half, then the up
// half.  Both passes are bound by HBM: every value is read and written once,
// a workgroup per row, 16 bytes a lane; arithmetic and the row's dot product
// are fp32.
#include "common.hpp"
#include "launch.hpp"

namespace moe {

namespace {

template <int V> struct Vec16 { typedef uint16_t type __attribute__((ext_vector_type(V))); };
template <> struct Vec16<1> { typedef uint16_t type; };

template <int V>
__device__ __forceinline__ void load_row(const uint16_t* p, float (&f)[V]) {
    const typename Vec16<V>::type v = *reinterpret_cast<const typename Vec16<V>::type*>(p);
    if constexpr (V == 1) f[0] = bf16_bits_to_f32(v);
    else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = bf16_bits_to_f32(v[i]);
    }
}

template <int V>
__device__ __forceinline__ void store_row(uint16_t* p, const float (&f)[V]) {
    if constexpr (V == 1) *p = f32_to_bf16_bits(f[0]);
    else {
        typename Vec16<V>::type v;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = f32_to_bf16_bits(f[i]);
        *reinterpret_cast<typename Vec16<V>::type*>(p) = v;
    }
}

// slot of row i: -1 padding, -2 a row past *num_rows (not touched)
__device__ __forceinline__ int gated_slot(const GatedArgs& a, int i) {
    if (a.num_rows && i >= *a.num_rows) return -2;
    if (!a.sorted) return i;
    const uint32_t p = (uint32_t)a.sorted[i];
    return p < a.slots ? (int)p : -1;
}

template <int V>
__global__ __launch_bounds__(256) void silu_mul_kernel(GatedArgs a) {
    const int i = (int)blockIdx.x;
    const int p = gated_slot(a, i);
    if (p == -2) return;
    const int n = ((int)blockIdx.y * 256 + (int)threadIdx.x) * V;
    if (n >= a.N) return;
    const uint16_t* g = a.g + (size_t)i * 2 * a.N + n;
    float y[V] = {};
    if (p >= 0) {
        const float w = a.weights ? a.weights[p] : 1.0f;
        float z[V], u[V];
        load_row<V>(g, z);
        load_row<V>(g + a.N, u);
#pragma unroll
        for (int v = 0; v < V; ++v) y[v] = w * silu(z[v]) * u[v];
    }
    store_row<V>(a.out + (size_t)i * a.N + n, y);
}

template <int V>
__global__ __launch_bounds__(256) void silu_mul_bwd_kernel(GatedArgs a) {
    __shared__ float part[4];
    const int i = (int)blockIdx.x;
    const int p = gated_slot(a, i);
    if (p == -2) return;
    const float w = p >= 0 && a.weights ? a.weights[p] : 1.0f;
    const uint16_t* g = a.g + (size_t)i * 2 * a.N;
    const uint16_t* d = a.da + (size_t)i * a.N;
    uint16_t* o = a.out + (size_t)i * 2 * a.N;
    float dot = 0.0f;
    for (int n = (int)threadIdx.x * V; n < a.N; n += 256 * V) {
        float dg[V] = {}, du[V] = {};
        if (p >= 0) {
            float z[V], u[V], da[V];
            load_row<V>(g + n, z);
            load_row<V>(g + a.N + n, u);
            load_row<V>(d + n, da);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float s = __builtin_amdgcn_rcpf(1.0f + __expf(-z[v]));
                const float act = z[v] * s;
                dot += da[v] * act * u[v];
                dg[v] = da[v] * w * u[v] * (s + act * (1.0f - s));
                du[v] = da[v] * w * act;
            }
        }
        store_row<V>(o + n, dg);
        store_row<V>(o + a.N + n, du);
    }
    if (!a.dweights || p < 0) return;  // the same for the whole workgroup
    dot = wave_sum_f32(dot);
    if (lane_id() == 0) part[threadIdx.x / kWave] = dot;
    __syncthreads();
    if (threadIdx.x == 0) a.dweights[p] = (part[0] + part[1]) + (part[2] + part[3]);
}

}  // namespace

void launch_silu_mul(const GatedArgs& a, hipStream_t s) {
    const int per = a.N % 8 == 0 ? 256 * 8 : 256;
    const dim3 grid(a.R, (a.N + per - 1) / per);
    if (a.N % 8 == 0) silu_mul_kernel<8><<<grid, 256, 0, s>>>(a);
    else silu_mul_kernel<1><<<grid, 256, 0, s>>>(a);
}

void launch_silu_mul_bwd(const GatedArgs& a, hipStream_t s) {
    if (a.N % 8 == 0) silu_mul_bwd_kernel<8><<<a.R, 256, 0, s>>>(a);
    else silu_mul_bwd_kernel<1><<<a.R, 256, 0, s>>>(a);
}

}  // namespace moe
