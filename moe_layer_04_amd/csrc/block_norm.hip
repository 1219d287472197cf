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
// Bound by HBM: a workgroup holds a whole row in registers (up to 16384 columns,
// the backward up to 8192), so each value is read and written once and the two
// sums of a row wait only for each other; longer rows are read again after a
// sum.  Statistics, sums over slots and gradients of the weights are fp32.  The
// weights' gradients are summed over a workgroup's rows, in registers (for
// longer rows in the partial row itself, read and written for every row),
// written as one partial row a workgroup and added up in a fixed order, so
// results do not depend on the order in which workgroups run.  4096 x 2 rows of
// 4096, fp32 stream: backward 74 + 4.7 us (369 MB, 5 TB/s; the second launch adds
// up the partial rows); 8 x 2 rows, bf16: forward 4.4 us, a launch and two
// barriers, backward 5.4 + 2.6.  4096 x 2 rows of 4096, bf16: forward 31.8 us with
// results that do not stay in the L2, 34.4 otherwise; the backward's are 77.3 us
// in ordinary stores, 78.0 so.
#include "common.hpp"
#include "launch.hpp"
#include "rows.hpp"

#include <type_traits>

namespace moe {

namespace {

constexpr int kNormThreads = 256 * 1024;  // of the backward's launch

// the residual stream's type
template <bool F32, bool ANY>
__device__ __forceinline__ void ld_h(const void* p, size_t at, int n, float (&f)[V]) {
    if constexpr (F32) ld_f32<ANY>((const float*)p + at, n, f);
    else ld_bf16<ANY>((const uint16_t*)p + at, n, f);
}
// stores f and leaves in it the value as stored
template <bool F32, bool ANY, bool ONCE>
__device__ __forceinline__ void st_h(void* p, size_t at, int n, float (&f)[V]) {
    if constexpr (F32) {
        st_f32<ANY, ONCE>((float*)p + at, n, f);
    } else {
        st_bf16<ANY, ONCE>((uint16_t*)p + at, n, f);
#pragma unroll
        for (int i = 0; i < V; ++i) f[i] = bf16_bits_to_f32(f32_to_bf16_bits(f[i]));
    }
}

// sum of a token's rows t*slots .. +slots at one column group
template <bool ANY>
__device__ __forceinline__ void ld_slots(const uint16_t* p, int t, int slots, int K, int col, int n,
                                         float (&f)[V]) {
    const uint16_t* q = p + (size_t)t * slots * K + col;
    ld_bf16<ANY>(q, n, f);
    for (int j = 1; j < slots; ++j) {
        float x[V];
        ld_bf16<ANY>(q + (size_t)j * K, n, x);
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
template <int TH, int C, bool F32, bool ANY>
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
            const int col = (c * TH + tid) * V, ci = C > 0 ? c : 0, n = ANY ? min(V, a.K - col) : V;
            if (col < a.K) {
                if constexpr (C > 0) ld_h<F32, ANY>(a.h, row + col, n, hh[ci]);
                ld_slots<ANY>(a.o, t, a.topk, a.K, col, n, f[ci]);
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
        const int col = (c * TH + tid) * V, ci = C > 0 ? c : 0, n = ANY ? min(V, a.K - col) : V;
        if (col >= a.K) continue;
        if (C == 0 || !a.o) ld_h<F32, ANY>(a.h, row + col, n, hh[ci]);
        if (a.o) {
            if constexpr (C == 0) ld_slots<ANY>(a.o, t, a.topk, a.K, col, n, f[ci]);
            float w[V];
            if (a.w_post) ld_f32<ANY>(a.w_post + col, n, w);
#pragma unroll
            for (int i = 0; i < V; ++i)
                hh[ci][i] += gs * (a.w_post ? f[ci][i] * r1 * w[i] : f[ci][i]);
            st_h<F32, ANY, (C > 0)>(a.h_out, row + col, n, hh[ci]);
        }
#pragma unroll
        for (int i = 0; i < V; ++i) ss += hh[ci][i] * hh[ci][i];
    }
    if (!a.w_pre) return;
    const float r2 = rsqrtf(block_sum<TH>(ss, part, half) * invk + a.eps);
    if (a.rstd_pre && tid == 0) a.rstd_pre[t] = r2;
    for (int c = 0; c < groups; ++c) {
        const int col = (c * TH + tid) * V, ci = C > 0 ? c : 0, n = ANY ? min(V, a.K - col) : V;
        if (col >= a.K) continue;
        // the thread's own columns, as it stored them
        if constexpr (C == 0) ld_h<F32, ANY>(a.o ? a.h_out : a.h, row + col, n, hh[ci]);
        float w[V], u[V];
        ld_f32<ANY>(a.w_pre + col, n, w);
#pragma unroll
        for (int i = 0; i < V; ++i) u[i] = hh[ci][i] * r2 * w[i];
        st_bf16<ANY, true>(a.u + row + col, n, u);
    }
}

// A workgroup takes the rows blockIdx.x, + gridDim.x, ...; partials: gridDim.x
// rows of K sums for dw_post, then as many for dw_pre (those that are asked
// for).
template <int TH, int C, bool F32, bool ANY>
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
    auto add = [&](float* p, int col, int n, const float (&v)[V], bool first) {
        float x[V];
        if (!first) ld_f32<ANY>(p + prow + col, n, x);
#pragma unroll
        for (int i = 0; i < V; ++i) x[i] = first ? v[i] : x[i] + v[i];
        st_f32<ANY>(p + prow + col, n, x);
    };
    for (int t = (int)blockIdx.x; t < a.M; t += (int)gridDim.x) {
        const bool first = t == (int)blockIdx.x;
        const size_t row = (size_t)t * a.K;
        const float gs = a.res_scale * (a.gate ? a.gate[t] : 1.0f);
        const float r1 = a.w_post ? a.rstd_post_in[t] : 1.0f;
        const float r2 = a.w_pre ? a.rstd_pre_in[t] : 1.0f;
        float dh[CR][V], hn[CR][V], z[CR][V];
        float s1 = 0.0f;
        // n and dn = du w_pre (kept in dh) of one group
        auto load_pre = [&](int ci, int col, int n, float (&du)[V]) {
            float w[V];
            ld_slots<ANY>(a.du, t, a.du_topk, a.K, col, n, du);
            ld_h<F32, ANY>(a.h, row + col, n, hn[ci]);
            ld_f32<ANY>(a.w_pre + col, n, w);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                hn[ci][i] *= r2;
                dh[ci][i] = du[i] * w[i];
            }
        };
        if (a.w_pre) {
            for (int c = 0; c < groups; ++c) {
                const int col = (c * TH + tid) * V, ci = C > 0 ? c : 0, n = ANY ? min(V, a.K - col) : V;
                if (col >= a.K) continue;
                float du[V];
                load_pre(ci, col, n, du);
                if constexpr (C > 0)
                    if (a.o) ld_slots<ANY>(a.o, t, a.topk, a.K, col, n, z[ci]);
                float dn[V];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    s1 += dh[ci][i] * hn[ci][i];
                    dn[i] = du[i] * hn[ci][i];
                }
                if constexpr (C > 0) {
#pragma unroll
                    for (int i = 0; i < V; ++i) sum_pre[ci][i] += dn[i];
                } else {
                    add(part_pre, col, n, dn, first);
                }
            }
            s1 = block_sum<TH>(s1, part, half) * invk;
        }
        float s2 = 0.0f;
        for (int c = 0; c < groups; ++c) {
            const int col = (c * TH + tid) * V, ci = C > 0 ? c : 0, n = ANY ? min(V, a.K - col) : V;
            if (col >= a.K) continue;
            float g[V] = {};
            if (a.dh_out) ld_h<F32, ANY>(a.dh_out, row + col, n, g);
            if (a.w_pre) {
                if constexpr (C == 0) {
                    float du[V];
                    load_pre(ci, col, n, du);
                }
#pragma unroll
                for (int i = 0; i < V; ++i) g[i] += r2 * (dh[ci][i] - hn[ci][i] * s1);
            }
#pragma unroll
            for (int i = 0; i < V; ++i) dh[ci][i] = g[i];
            if constexpr (F32) st_f32<ANY>((float*)a.h_out + row + col, n, g);
            else st_bf16<ANY>((uint16_t*)a.h_out + row + col, n, g);
            if (!a.o) continue;
            if (C == 0 || !a.w_pre) ld_slots<ANY>(a.o, t, a.topk, a.K, col, n, z[ci]);
            float w[V], dz[V];
            if (a.w_post) ld_f32<ANY>(a.w_post + col, n, w);
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
                add(part_post, col, n, dz, first);
            }
        }
        if (!a.o) continue;
        if (a.w_post || a.dgate) s2 = block_sum<TH>(s2, part, half);
        if (a.dgate && tid == 0) a.dgate[t] = a.res_scale * s2;
        s2 *= invk;
        for (int c = 0; c < groups; ++c) {
            const int col = (c * TH + tid) * V, ci = C > 0 ? c : 0, n = ANY ? min(V, a.K - col) : V;
            if (col >= a.K) continue;
            if constexpr (C == 0) {
                // b and z again: dh from its inputs, not from its rounding
                float g[V] = {}, w[V];
                if (a.dh_out) ld_h<F32, ANY>(a.dh_out, row + col, n, g);
                if (a.w_pre) {
                    float du[V];
                    load_pre(ci, col, n, du);
#pragma unroll
                    for (int i = 0; i < V; ++i) g[i] += r2 * (dh[ci][i] - hn[ci][i] * s1);
                }
                ld_slots<ANY>(a.o, t, a.topk, a.K, col, n, z[ci]);
                if (a.w_post) ld_f32<ANY>(a.w_post + col, n, w);
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
            st_bf16<ANY>(a.u + row + col, n, y);
        }
    }
    if constexpr (C > 0) {
        for (int c = 0; c < groups; ++c) {
            const int col = (c * TH + tid) * V, n = ANY ? min(V, a.K - col) : V;
            if (col >= a.K) continue;
            if (part_post) st_f32<ANY>(part_post + prow + col, n, sum_post[c]);
            if (part_pre) st_f32<ANY>(part_pre + prow + col, n, sum_pre[c]);
        }
    }
}

// dw[k] = sum of the partial rows: 32 columns a workgroup, 32 threads a column
// each adding every 32nd row in ascending order, then the 32 sums in order
constexpr int kPartCols = 32, kPartRows = 32;
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

// Threads and column groups that hold a row of K columns in registers; longer
// rows are re-read.
// The backward holds five rows of values and two of sums: one group a thread
// (126 registers, four waves a SIMD) took 74 us where two groups with half the
// threads (194 registers, two waves) took 87 (4096 rows of 4096, two slots,
// fp32 stream: 385 MB).  1024 threads are one workgroup a CU, which nothing runs
// beside at its two barriers a row, and with a bf16 stream or odd widths 2 to 6
// registers short: 4096 x 2 rows of 5120, 7168 and 8192, bf16 94, 110 and 119 us
// (the bytes' floor 70, 98 and 112), fp32 107, 135 and 151 (96, 134 and 154).
// Re-read rows: 1024 x 2 of 16384, bf16 127 us (56), fp32 155 (77).  Widths that
// are no multiples of 8, three waves a SIMD: 4096 x 2 rows of 4095 190 us (56 and
// 77).
template <int TH, int C>
struct Shape {
    static constexpr int kThreads = TH, kGroups = C;
};
template <bool BWD, typename F>
void pick_shape(int K, const F& f) {
    if (K <= 512) return f(Shape<64, 1>{});
    if (K <= 1024) return f(Shape<128, 1>{});
    if (K <= 2048) return f(Shape<256, 1>{});
    if constexpr (BWD) {
        if (K <= 4096) return f(Shape<512, 1>{});
        if (K <= 8192) return f(Shape<1024, 1>{});
    } else {
        if (K <= 4096) return f(Shape<256, 2>{});
        if (K <= 8192) return f(Shape<512, 2>{});
        if (K <= 16384) return f(Shape<1024, 2>{});
    }
    f(Shape<512, 0>{});
}

template <typename F>
void with_types(const NormArgs& a, const F& run) {
    if (a.K % V == 0) {
        if (a.h_f32) run(std::true_type{}, std::false_type{});
        else run(std::false_type{}, std::false_type{});
    } else {
        if (a.h_f32) run(std::true_type{}, std::true_type{});
        else run(std::false_type{}, std::true_type{});
    }
}

// Workgroups of the backward, each with one partial row of either gradient:
// 1024 threads a CU.
int norm_parts(int M, int K) {
    int parts = 0;
    pick_shape<true>(K, [&](auto shape) { parts = kNormThreads / shape.kThreads; });
    return M < parts ? M : parts;
}

}  // namespace

void launch_block_norm(const NormArgs& a, hipStream_t s) {
    pick_shape<false>(a.K, [&](auto shape) {
        constexpr int TH = shape.kThreads, C = shape.kGroups;
        auto run = [&](auto f32, auto any) {
            block_norm_kernel<TH, C, decltype(f32)::value, decltype(any)::value><<<a.M, TH, 0, s>>>(a);
        };
        with_types(a, run);
    });
}

// partial rows of both weights' gradients
size_t block_norm_bwd_workspace(int M, int K) { return (size_t)norm_parts(M, K) * K * 4 * 2; }

void launch_block_norm_bwd(const NormArgs& a, float* partials, hipStream_t s) {
    const int parts = norm_parts(a.M, a.K);
    float* post = a.w_post ? partials : nullptr;
    float* pre = a.w_pre ? partials + (a.w_post ? (size_t)parts * a.K : 0) : nullptr;
    if (parts)
        pick_shape<true>(a.K, [&](auto shape) {
            constexpr int TH = shape.kThreads, C = shape.kGroups;
            auto run = [&](auto f32, auto any) {
                block_norm_bwd_kernel<TH, C, decltype(f32)::value, decltype(any)::value>
                    <<<parts, TH, 0, s>>>(a, post, pre);
            };
            with_types(a, run);
        });
    if (post || pre)
        norm_parts_kernel<<<dim3((a.K + kPartCols - 1) / kPartCols, 2), kPartCols * kPartRows, 0, s>>>(
            post, pre, parts, a.K, a.dw_post, a.dw_pre);
}

}  // namespace moe
