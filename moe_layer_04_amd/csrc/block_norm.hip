// block_norm.hip -- the norms on both sides of a block of the network, with
// the block's gate and the residual scale, as one pass over a token's row:
//
//   o     = sum_j o[t,j]                       (a token's slots, fp32)
//   z     = o / rms(o),  rms(v)^2 = mean(v^2) + eps
//   h'    = h + s gate[t] z w_post             (kept in h's type)
//   u     = h' / rms(h') w_pre                 (what the next block reads)
//
// Without w_post the block's output is added as it is (z = o); without o only
// the second norm is taken; without w_pre only h' is formed.  Backward, with
// n = h' rstd_pre, c = du w_pre, b = dh w_post:
//
//   dh    = dh' + rstd_pre (c - n mean(c n))
//   do    = s gate rstd_post (b - z mean(b z)),   dgate = s sum(b z)
//   dw_post = sum_t s gate dh z,                  dw_pre = sum_t du n
//
// Bound by HBM: a workgroup holds a whole row in registers, so each value is
// read and written once and the two sums of a row wait only for each other.
// Statistics, sums over slots and gradients of the weights are fp32.  The
// weights' gradients are summed over a workgroup's rows in registers, written
// as one partial row a workgroup and added up in a fixed order, so results do
// not depend on the order in which workgroups run.
#include "common.hpp"
#include "launch.hpp"

#include <type_traits>

namespace moe {

namespace {

constexpr int kNormMaxParts = 512;  // workgroups of the backward = partial rows

template <int V> struct Bits { typedef uint16_t type __attribute__((ext_vector_type(V))); };
template <> struct Bits<1> { typedef uint16_t type; };
template <int V> struct Fp { typedef float type __attribute__((ext_vector_type(V))); };
template <> struct Fp<1> { typedef float type; };

template <int V>
__device__ __forceinline__ void ld_bf16(const uint16_t* p, float (&f)[V]) {
    const typename Bits<V>::type v = *reinterpret_cast<const typename Bits<V>::type*>(p);
    if constexpr (V == 1) f[0] = bf16_bits_to_f32(v);
    else {
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = bf16_bits_to_f32(v[i]);
    }
}
template <int V>
__device__ __forceinline__ void st_bf16(uint16_t* p, const float (&f)[V]) {
    if constexpr (V == 1) *p = f32_to_bf16_bits(f[0]);
    else {
        typename Bits<V>::type v;
#pragma unroll
        for (int i = 0; i < V; ++i) v[i] = f32_to_bf16_bits(f[i]);
        *reinterpret_cast<typename Bits<V>::type*>(p) = v;
    }
}
template <int V>
__device__ __forceinline__ void ld_f32(const float* p, float (&f)[V]) {
    if constexpr (V == 1) f[0] = *p;
    else {
#pragma unroll
        for (int i = 0; i < V; i += 4) {
            const f32x4_t v = *reinterpret_cast<const f32x4_t*>(p + i);
#pragma unroll
            for (int j = 0; j < 4; ++j) f[i + j] = v[j];
        }
    }
}
template <int V>
__device__ __forceinline__ void st_f32(float* p, const float (&f)[V]) {
    if constexpr (V == 1) *p = f[0];
    else {
#pragma unroll
        for (int i = 0; i < V; i += 4)
            *reinterpret_cast<f32x4_t*>(p + i) = f32x4_t{f[i], f[i + 1], f[i + 2], f[i + 3]};
    }
}
// the residual stream's type
template <int V, bool F32>
__device__ __forceinline__ void ld_h(const void* p, size_t at, float (&f)[V]) {
    if constexpr (F32) ld_f32<V>((const float*)p + at, f);
    else ld_bf16<V>((const uint16_t*)p + at, f);
}
// stores f and leaves in it the value as stored
template <int V, bool F32>
__device__ __forceinline__ void st_h(void* p, size_t at, float (&f)[V]) {
    if constexpr (F32) {
        st_f32<V>((float*)p + at, f);
    } else {
        st_bf16<V>((uint16_t*)p + at, f);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = bf16_bits_to_f32(f32_to_bf16_bits(f[i]));
    }
}

// sum of a token's rows t*slots .. +slots at one column group
template <int V>
__device__ __forceinline__ void ld_slots(const uint16_t* p, int t, int slots, int K, int col,
                                         float (&f)[V]) {
    const uint16_t* q = p + (size_t)t * slots * K + col;
    ld_bf16<V>(q, f);
    for (int j = 1; j < slots; ++j) {
        float x[V];
        ld_bf16<V>(q + (size_t)j * K, x);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] += x[i];
    }
}

// Sum over the workgroup, in every thread.  Successive calls alternate the
// two halves of `part`: the barrier of a call separates the reads of the call
// before it from the writes of the call after it.
template <int TH>
__device__ __forceinline__ float block_sum(float v, float (&part)[2][16], int& half) {
    v = wave_sum_f32(v);
    if constexpr (TH == kWave) return v;
    float* p = part[half];
    half ^= 1;
    if (lane_id() == 0) p[threadIdx.x / kWave] = v;
    __syncthreads();
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < TH / kWave; ++i) s += p[i];
    return s;
}

// C > 0: a thread keeps its C groups of V columns in registers (K <= TH*V*C);
// C == 0: rows of any length, re-read between the passes.
template <int TH, int V, int C, bool F32>
__global__ __launch_bounds__(TH) void block_norm_kernel(NormArgs a) {
    __shared__ float part[2][16];
    int half = 0;
    const int t = (int)blockIdx.x;
    const int tid = (int)threadIdx.x;
    const float invk = 1.0f / (float)a.K;
    const size_t row = (size_t)t * a.K;
    const float gs = a.o ? a.res_scale * (a.gate ? a.gate[t] : 1.0f) : 0.0f;
    constexpr int CR = C > 0 ? C : 1;
    const int groups = C > 0 ? C : (a.K + TH * V - 1) / (TH * V);
    float f[CR][V], hh[CR][V];
    float r1 = 1.0f;
    if (a.o) {
        float ss = 0.0f;
        for (int c = 0; c < groups; ++c) {
            const int col = (c * TH + tid) * V, ci = C > 0 ? c : 0;
            if (col < a.K) {
                if constexpr (C > 0) ld_h<V, F32>(a.h, row + col, hh[ci]);
                ld_slots<V>(a.o, t, a.topk, a.K, col, f[ci]);
#pragma unroll
                for (int i = 0; i < V; ++i) ss += f[ci][i] * f[ci][i];
            }
        }
        if (a.w_post) {
            r1 = rsqrtf(block_sum<TH>(ss, part, half) * invk + a.eps);
            if (a.rstd_post && tid == 0) a.rstd_post[t] = r1;
        }
    }
    float ss = 0.0f;
    for (int c = 0; c < groups; ++c) {
        const int col = (c * TH + tid) * V, ci = C > 0 ? c : 0;
        if (col >= a.K) continue;
        if (C == 0 || !a.o) ld_h<V, F32>(a.h, row + col, hh[ci]);
        if (a.o) {
            if constexpr (C == 0) ld_slots<V>(a.o, t, a.topk, a.K, col, f[ci]);
            float w[V];
            if (a.w_post) ld_f32<V>(a.w_post + col, w);
#pragma unroll
            for (int i = 0; i < V; ++i)
                hh[ci][i] += gs * (a.w_post ? f[ci][i] * r1 * w[i] : f[ci][i]);
            st_h<V, F32>(a.h_out, row + col, hh[ci]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) ss += hh[ci][i] * hh[ci][i];
    }
    if (!a.w_pre) return;
    const float r2 = rsqrtf(block_sum<TH>(ss, part, half) * invk + a.eps);
    if (a.rstd_pre && tid == 0) a.rstd_pre[t] = r2;
    for (int c = 0; c < groups; ++c) {
        const int col = (c * TH + tid) * V, ci = C > 0 ? c : 0;
        if (col >= a.K) continue;
        // the thread's own columns, as it stored them
        if constexpr (C == 0) ld_h<V, F32>(a.o ? a.h_out : a.h, row + col, hh[ci]);
        float w[V], u[V];
        ld_f32<V>(a.w_pre + col, w);
#pragma unroll
        for (int i = 0; i < V; ++i) u[i] = hh[ci][i] * r2 * w[i];
        st_bf16<V>(a.u + row + col, u);
    }
}

// A workgroup takes the rows blockIdx.x, + gridDim.x, ...; partials: gridDim.x
// rows of K sums for dw_post, then as many for dw_pre (those that are asked
// for).
template <int TH, int V, int C, bool F32>
__global__ __launch_bounds__(TH) void block_norm_bwd_kernel(NormArgs a, float* part_post,
                                                            float* part_pre) {
    __shared__ float part[2][16];
    int half = 0;
    const int tid = (int)threadIdx.x;
    const float invk = 1.0f / (float)a.K;
    constexpr int CR = C > 0 ? C : 1;
    const int groups = C > 0 ? C : (a.K + TH * V - 1) / (TH * V);
    float sum_post[CR][V] = {}, sum_pre[CR][V] = {};
    const size_t prow = (size_t)blockIdx.x * a.K;
    auto add = [&](float* p, int col, const float (&v)[V], bool first) {
        float x[V];
        if (!first) ld_f32<V>(p + prow + col, x);
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = first ? v[i] : x[i] + v[i];
        st_f32<V>(p + prow + col, x);
    };
    for (int t = (int)blockIdx.x; t < a.M; t += (int)gridDim.x) {
        const bool first = t == (int)blockIdx.x;
        const size_t row = (size_t)t * a.K;
        const float gs = a.res_scale * (a.gate ? a.gate[t] : 1.0f);
        const float r1 = a.w_post ? a.rstd_post_in[t] : 1.0f;
        const float r2 = a.w_pre ? a.rstd_pre_in[t] : 1.0f;
        float dh[CR][V], n[CR][V], z[CR][V];
        float s1 = 0.0f;
        // n and dn = du w_pre (kept in dh) of one group
        auto load_pre = [&](int ci, int col, float (&du)[V]) {
            float w[V];
            ld_slots<V>(a.du, t, a.du_topk, a.K, col, du);
            ld_h<V, F32>(a.h, row + col, n[ci]);
            ld_f32<V>(a.w_pre + col, w);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                n[ci][i] *= r2;
                dh[ci][i] = du[i] * w[i];
            }
        };
        if (a.w_pre) {
            for (int c = 0; c < groups; ++c) {
                const int col = (c * TH + tid) * V, ci = C > 0 ? c : 0;
                if (col >= a.K) continue;
                float du[V];
                load_pre(ci, col, du);
                if constexpr (C > 0)
                    if (a.o) ld_slots<V>(a.o, t, a.topk, a.K, col, z[ci]);
                float dn[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    s1 += dh[ci][i] * n[ci][i];
                    dn[i] = du[i] * n[ci][i];
                }
                if constexpr (C > 0) {
#pragma unroll
                    for (int i = 0; i < V; ++i) sum_pre[ci][i] += dn[i];
                } else {
                    add(part_pre, col, dn, first);
                }
            }
            s1 = block_sum<TH>(s1, part, half) * invk;
        }
        float s2 = 0.0f;
        for (int c = 0; c < groups; ++c) {
            const int col = (c * TH + tid) * V, ci = C > 0 ? c : 0;
            if (col >= a.K) continue;
            float g[V] = {};
            if (a.dh_out) ld_h<V, F32>(a.dh_out, row + col, g);
            if (a.w_pre) {
                if constexpr (C == 0) {
                    float du[V];
                    load_pre(ci, col, du);
                }
#pragma unroll
                for (int i = 0; i < V; ++i) g[i] += r2 * (dh[ci][i] - n[ci][i] * s1);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) dh[ci][i] = g[i];
            if constexpr (F32) st_f32<V>((float*)a.h_out + row + col, g);
            else st_bf16<V>((uint16_t*)a.h_out + row + col, g);
            if (!a.o) continue;
            if (C == 0 || !a.w_pre) ld_slots<V>(a.o, t, a.topk, a.K, col, z[ci]);
            float w[V], dz[V];
            if (a.w_post) ld_f32<V>(a.w_post + col, w);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                z[ci][i] *= r1;
                dz[i] = gs * dh[ci][i] * z[ci][i];
                dh[ci][i] = a.w_post ? dh[ci][i] * w[i] : dh[ci][i];
                s2 += dh[ci][i] * z[ci][i];
            }
            if (!a.w_post) continue;
            if constexpr (C > 0) {
#pragma unroll
                for (int i = 0; i < V; ++i) sum_post[ci][i] += dz[i];
            } else {
                add(part_post, col, dz, first);
            }
        }
        if (!a.o) continue;
        if (a.w_post || a.dgate) s2 = block_sum<TH>(s2, part, half);
        if (a.dgate && tid == 0) a.dgate[t] = a.res_scale * s2;
        s2 *= invk;
        for (int c = 0; c < groups; ++c) {
            const int col = (c * TH + tid) * V, ci = C > 0 ? c : 0;
            if (col >= a.K) continue;
            if constexpr (C == 0) {
                // b and z again: dh from its inputs, not from its rounding
                float g[V] = {}, w[V];
                if (a.dh_out) ld_h<V, F32>(a.dh_out, row + col, g);
                if (a.w_pre) {
                    float du[V];
                    load_pre(ci, col, du);
#pragma unroll
                    for (int i = 0; i < V; ++i) g[i] += r2 * (dh[ci][i] - n[ci][i] * s1);
                }
                ld_slots<V>(a.o, t, a.topk, a.K, col, z[ci]);
                if (a.w_post) ld_f32<V>(a.w_post + col, w);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    z[ci][i] *= r1;
                    dh[ci][i] = a.w_post ? g[i] * w[i] : g[i];
                }
            }
            float y[V];
#pragma unroll
            for (int i = 0; i < V; ++i)
                y[i] = gs * (a.w_post ? r1 * (dh[ci][i] - z[ci][i] * s2) : dh[ci][i]);
            st_bf16<V>(a.u + row + col, y);
        }
    }
    if constexpr (C > 0) {
        for (int c = 0; c < groups; ++c) {
            const int col = (c * TH + tid) * V;
            if (col >= a.K) continue;
            if (part_post) st_f32<V>(part_post + prow + col, sum_post[c]);
            if (part_pre) st_f32<V>(part_pre + prow + col, sum_pre[c]);
        }
    }
}

// dw[k] = sum of the partial rows: 32 columns a workgroup, 16 threads a column
// each adding every 16th row in ascending order, then the 16 sums in order
constexpr int kPartCols = 32, kPartRows = 16;
__global__ __launch_bounds__(kPartCols * kPartRows) void norm_parts_kernel(
    const float* post, const float* pre, int parts, int K, float* dw_post, float* dw_pre) {
    __shared__ float sums[kPartRows][kPartCols];
    const float* src = blockIdx.y ? pre : post;
    float* dst = blockIdx.y ? dw_pre : dw_post;
    if (!dst) return;
    const int c = (int)threadIdx.x % kPartCols, q = (int)threadIdx.x / kPartCols;
    const int col = (int)blockIdx.x * kPartCols + c;
    float s = 0.0f;
    if (col < K) {
        int p = q;
        for (; p + 7 * kPartRows < parts; p += 8 * kPartRows) {
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = src[(size_t)(p + i * kPartRows) * K + col];
#pragma unroll
            for (int i = 0; i < 8; ++i) s += v[i];
        }
        for (; p < parts; p += kPartRows) s += src[(size_t)p * K + col];
    }
    sums[q][c] = s;
    __syncthreads();
    if (q == 0 && col < K) {
#pragma unroll
        for (int i = 1; i < kPartRows; ++i) s += sums[i][c];
        dst[col] = s;
    }
}

// Threads, columns per load and column groups that hold a row of K columns in
// registers; rows that are no multiple of 8 long, or too long, are re-read.
template <int TH, int V, int C>
struct Shape {
    static constexpr int kThreads = TH, kVec = V, kGroups = C;
};
template <bool BWD, typename F>
void pick_shape(int K, const F& f) {
    if (K % 8 || K > 16384) f(Shape<256, 1, 0>{});
    else if (K <= 512) f(Shape<64, 8, 1>{});
    else if (K <= 2048) f(Shape<256, 8, 1>{});
    else if (K <= 4096) f(Shape<256, 8, 2>{});
    else if (K <= 8192) f(Shape<512, 8, 2>{});
    // the backward's five rows of values fit 512 threads' registers, not 1024's
    else if constexpr (BWD) f(Shape<512, 8, 4>{});
    else f(Shape<1024, 8, 2>{});
}

int norm_parts(int M) { return M < kNormMaxParts ? M : kNormMaxParts; }

}  // namespace

void launch_block_norm(const NormArgs& a, hipStream_t s) {
    pick_shape<false>(a.K, [&](auto shape) {
        constexpr int TH = shape.kThreads, V = shape.kVec, C = shape.kGroups;
        if (a.h_f32) block_norm_kernel<TH, V, C, true><<<a.M, TH, 0, s>>>(a);
        else block_norm_kernel<TH, V, C, false><<<a.M, TH, 0, s>>>(a);
    });
}

size_t block_norm_bwd_workspace(int M, int K, bool post, bool pre) {
    return (size_t)norm_parts(M) * K * 4 * ((post ? 1 : 0) + (pre ? 1 : 0));
}

void launch_block_norm_bwd(const NormArgs& a, float* partials, hipStream_t s) {
    const int parts = norm_parts(a.M);
    float* post = a.w_post ? partials : nullptr;
    float* pre = a.w_pre ? partials + (a.w_post ? (size_t)parts * a.K : 0) : nullptr;
    if (parts)
        pick_shape<true>(a.K, [&](auto shape) {
            constexpr int TH = shape.kThreads, V = shape.kVec, C = shape.kGroups;
            if (a.h_f32) block_norm_bwd_kernel<TH, V, C, true><<<parts, TH, 0, s>>>(a, post, pre);
            else block_norm_bwd_kernel<TH, V, C, false><<<parts, TH, 0, s>>>(a, post, pre);
        });
    if (post || pre)
        norm_parts_kernel<<<dim3((a.K + kPartCols - 1) / kPartCols, 2), kPartCols * kPartRows, 0, s>>>(
            post, pre, parts, a.K, a.dw_post, a.dw_pre);
}

}  // namespace moe
