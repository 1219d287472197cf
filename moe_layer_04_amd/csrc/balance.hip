// balance.hip -- the balance loss of the router, the counts behind it, and the
// gradient of the logits.  V: the tokens that count (mask), n of them;
// p_t = softmax(l_t); c_e: slots of V's tokens that picked expert e:
//
//   f_e = c_e / (n k),   P_e = sum_{t in V} p_te / n,   loss = E sum_e f_e P_e
//   dl_te = dloss E / n  p_te (f_e - sum_i p_ti f_i),   zero rows outside V
//
// L lanes share a token, four experts each (L: the least power of two that
// holds E), so a wave takes 64 / L tokens, and a token's maximum and sums stay
// within its lanes.  Both passes are bound by HBM: the logits are read once, as 16
// bytes a lane.  Sums are fp32 in a fixed order: a lane's tokens one after the
// other, then the lanes, the waves and the workgroups; counts are integers.
#include "common.hpp"
#include "launch.hpp"

#include <type_traits>

namespace moe {

namespace {

constexpr int kSplit = 4;  // experts a lane

template <int L, typename F>
__device__ __forceinline__ float group_reduce(float v, F f) {
    if constexpr (L > 1) v = f(v, __uint_as_float(xchg_u32<0>(__float_as_uint(v))));
    if constexpr (L > 2) v = f(v, __uint_as_float(xchg_u32<1>(__float_as_uint(v))));
    if constexpr (L > 4) v = f(v, __uint_as_float(xchg_u32<2>(__float_as_uint(v))));
    if constexpr (L > 8) v = f(v, __uint_as_float(xchg_u32<3>(__float_as_uint(v))));
    if constexpr (L > 16) v = f(v, __uint_as_float(xchg_u32<4>(__float_as_uint(v))));
    if constexpr (L > 32)
        v = f(__uint_as_float(readlane_u32(__float_as_uint(v), 0)),
              __uint_as_float(readlane_u32(__float_as_uint(v), 32)));
    return v;
}
template <int L>
__device__ __forceinline__ float group_sum(float v) {
    return group_reduce<L>(v, [](float a, float b) { return a + b; });
}
template <int L>
__device__ __forceinline__ float group_max(float v) {
    return group_reduce<L>(v, [](float a, float b) { return fmaxf(a, b); });
}

// This lane's four logits; -inf past the last expert
template <bool VEC>
__device__ __forceinline__ f32x4_t ld_logits(const float* row, int e, int E) {
    if constexpr (VEC) {
        if (e < E) return *reinterpret_cast<const f32x4_t*>(row + e);
    }
    f32x4_t v;
#pragma unroll
    for (int i = 0; i < kSplit; ++i) v[i] = !VEC && e + i < E ? row[e + i] : -__builtin_inff();
    return v;
}

// Probabilities of a token from its lanes' logits; zeros where all are -inf
// (a NaN makes all of them NaN).
template <int L>
__device__ __forceinline__ f32x4_t probabilities(f32x4_t l) {
    float m = fmaxf(fmaxf(l[0], l[1]), fmaxf(l[2], l[3]));
    m = group_max<L>(m);
    const float base = m == -__builtin_inff() ? 0.0f : m;
    f32x4_t p;
#pragma unroll
    for (int i = 0; i < kSplit; ++i) p[i] = __expf(l[i] - base);
    const float s = group_sum<L>((p[0] + p[1]) + (p[2] + p[3]));
    const float r = s == 0.0f ? 0.0f : 1.0f / s;
#pragma unroll
    for (int i = 0; i < kSplit; ++i) p[i] *= r;
    return p;
}

// loss, counts, tokens and probs from the sums of all tokens, by threads
// 0..255 of a workgroup (thread e: expert e)
__device__ __forceinline__ void balance_finish(const BalanceArgs& a, float psum, int count, int n,
                                               float (&part)[4]) {
    const int e = (int)threadIdx.x;
    float term = 0.0f;
    if (e < a.E) {
        const float inv = n > 0 ? 1.0f / (float)n : 0.0f;
        const float P = psum * inv;
        a.counts[e] = count;
        a.probs[e] = P;
        term = (float)count * inv / (float)a.topk * P;
    }
    if (e == 0) a.tokens[0] = n;
    term = wave_sum_f32(term);
    if (e < 256 && lane_id() == 0) part[e / kWave] = term;
    __syncthreads();
    if (e == 0) a.loss[0] = (float)a.E * ((part[0] + part[1]) + (part[2] + part[3]));
}

// A workgroup takes the tokens [b, b + 1) * per; with more than one of them
// each leaves its sums in the workspace, [groups][E] of p, then of counts, then
// [groups] of tokens.
template <int L, bool VEC>
__global__ __launch_bounds__(256) void balance_kernel(BalanceArgs a, int per, float* __restrict__ psums,
                                                      int* __restrict__ csums, int* __restrict__ tsums) {
    __shared__ float sums[4][256];
    __shared__ int hist[256];
    __shared__ int seen[4];
    __shared__ float part[4];
    constexpr int TW = kWave / L;  // tokens a wave
    const int tid = (int)threadIdx.x, lane = lane_id(), wave = tid / kWave;
    const int first = (int)blockIdx.x * per, last = min(first + per, a.M);
    const int e0 = (lane % L) * kSplit;
    hist[tid] = 0;
    __syncthreads();
    f32x4_t acc = {0, 0, 0, 0};
    int tokens = 0;
    for (int t0 = first + wave * TW; t0 < last; t0 += 4 * TW) {
        const int t = t0 + lane / L;
        const bool in = t < last && (!a.mask || a.mask[t]);
        tokens += in && lane % L == 0;
        f32x4_t l = {0, 0, 0, 0};
        if (in) l = ld_logits<VEC>(a.logits + (size_t)t * a.E, e0, a.E);
        const f32x4_t p = probabilities<L>(l);
        if (in) acc += p;
    }
    const long s0 = (long)first * a.topk, s1 = (long)last * a.topk;
    for (long s = s0 + tid; s < s1; s += 256) {
        const uint32_t e = (uint32_t)a.ids[s];
        if (e < (uint32_t)a.E && (!a.mask || a.mask[s / a.topk])) atomicAdd(&hist[e], 1);
    }
    // lanes with the same experts, then the waves
#pragma unroll
    for (int i = 0; i < kSplit; ++i) {
        float v = acc[i];
#pragma unroll
        for (int d = L; d < kWave; d *= 2) v += __shfl_xor(v, d);
        if (lane < L) sums[wave][e0 + i] = v;
    }
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) tokens += __shfl_xor(tokens, d);
    if (lane == 0) seen[wave] = tokens;
    __syncthreads();
    const float psum = tid < L * kSplit ? (sums[0][tid] + sums[1][tid]) + (sums[2][tid] + sums[3][tid]) : 0.0f;
    const int n = (seen[0] + seen[1]) + (seen[2] + seen[3]);
    if (gridDim.x == 1) {
        balance_finish(a, psum, hist[tid], n, part);
        return;
    }
    if (tid < a.E) {
        psums[(size_t)blockIdx.x * a.E + tid] = psum;
        csums[(size_t)blockIdx.x * a.E + tid] = hist[tid];
    }
    if (tid == 0) tsums[blockIdx.x] = n;
}

// the workgroups' sums in order: four threads an expert take a quarter of them each
__global__ __launch_bounds__(1024) void balance_join_kernel(BalanceArgs a, int groups,
                                                            const float* __restrict__ psums,
                                                            const int* __restrict__ csums,
                                                            const int* __restrict__ tsums) {
    __shared__ float ps[4][256];
    __shared__ int cs[4][256], ts[4];
    __shared__ float part[4];
    const int tid = (int)threadIdx.x, e = tid % 256, q = tid / 256;
    const int per = (groups + 3) / 4, from = q * per, to = min(from + per, groups);
    float p = 0.0f;
    int c = 0, n = 0;
    if (e < a.E) {
#pragma unroll 8
        for (int g = from; g < to; ++g) {
            p += psums[(size_t)g * a.E + e];
            c += csums[(size_t)g * a.E + e];
        }
    }
    ps[q][e] = p;
    cs[q][e] = c;
    if (tid < 256) {
        for (int g = tid; g < groups; g += 256) n += tsums[g];
#pragma unroll
        for (int d = 1; d < kWave; d *= 2) n += __shfl_xor(n, d);
        if (lane_id() == 0) ts[tid / kWave] = n;
    }
    __syncthreads();
    balance_finish(a, (ps[0][e] + ps[1][e]) + (ps[2][e] + ps[3][e]),
                   (cs[0][e] + cs[1][e]) + (cs[2][e] + cs[3][e]), (ts[0] + ts[1]) + (ts[2] + ts[3]), part);
}

template <int L, bool VEC>
__global__ __launch_bounds__(256) void balance_bwd_kernel(BalanceArgs a) {
    constexpr int TW = kWave / L;
    const int lane = lane_id(), e0 = (lane % L) * kSplit;
    const int n = a.tokens[0];
    const float inv = n > 0 ? 1.0f / (float)n : 0.0f;
    f32x4_t f;
#pragma unroll
    for (int i = 0; i < kSplit; ++i)
        f[i] = e0 + i < a.E ? (float)a.counts[e0 + i] * inv / (float)a.topk : 0.0f;
    const float up = a.dloss[0] * (float)a.E * inv;
    const long stride = (long)gridDim.x * 4 * TW;
    for (long t0 = ((long)blockIdx.x * 4 + threadIdx.x / kWave) * TW; t0 < a.M; t0 += stride) {
        const long t = t0 + lane / L;
        const bool in = t < a.M, counts = in && (!a.mask || a.mask[t]);
        f32x4_t l = {0, 0, 0, 0};
        if (counts) l = ld_logits<VEC>(a.logits + (size_t)t * a.E, e0, a.E);
        f32x4_t p = probabilities<L>(l);
        const float dot = group_sum<L>((p[0] * f[0] + p[1] * f[1]) + (p[2] * f[2] + p[3] * f[3]));
#pragma unroll
        for (int i = 0; i < kSplit; ++i) p[i] = counts && n > 0 ? up * p[i] * (f[i] - dot) : 0.0f;
        if (!in) continue;
        float* o = a.dlogits + (size_t)t * a.E + e0;
        if constexpr (VEC) {
            if (e0 < a.E) *reinterpret_cast<f32x4_t*>(o) = p;
        } else {
#pragma unroll
            for (int i = 0; i < kSplit; ++i)
                if (e0 + i < a.E) o[i] = p[i];
        }
    }
}

// calls f(lanes a token, whether rows are whole vectors)
template <typename F>
void by_experts(int E, F f) {
    auto vec = [&](auto lanes) {
        if (E % kSplit == 0) f(lanes, std::true_type{});
        else f(lanes, std::false_type{});
    };
    if (E <= 4) vec(std::integral_constant<int, 1>{});
    else if (E <= 8) vec(std::integral_constant<int, 2>{});
    else if (E <= 16) vec(std::integral_constant<int, 4>{});
    else if (E <= 32) vec(std::integral_constant<int, 8>{});
    else if (E <= 64) vec(std::integral_constant<int, 16>{});
    else if (E <= 128) vec(std::integral_constant<int, 32>{});
    else vec(std::integral_constant<int, 64>{});
}

// Tokens a workgroup: at least 32 rounds of its waves' loads' worth of values,
// and no more than 256 workgroups.
int balance_per(int M, int E) {
    int per = (8192 + E - 1) / E;
    if (per < (M + 255) / 256) per = (M + 255) / 256;
    return per;
}
int balance_groups(int M, int E) { return M == 0 ? 1 : (M + balance_per(M, E) - 1) / balance_per(M, E); }

}  // namespace

size_t balance_workspace(int M, int E) {
    const int groups = balance_groups(M, E);
    return groups > 1 ? (size_t)groups * (2 * E + 1) * 4 : 0;
}

void launch_balance(const BalanceArgs& a, void* workspace, hipStream_t s) {
    const int groups = balance_groups(a.M, a.E), per = balance_per(a.M, a.E);
    float* psums = (float*)workspace;
    int* csums = (int*)workspace + (size_t)groups * a.E;
    int* tsums = csums + (size_t)groups * a.E;
    by_experts(a.E, [&](auto lanes, auto vec) {
        balance_kernel<decltype(lanes)::value, decltype(vec)::value><<<groups, 256, 0, s>>>(a, per, psums, csums,
                                                                                           tsums);
    });
    if (groups > 1) balance_join_kernel<<<1, 1024, 0, s>>>(a, groups, psums, csums, tsums);
}

void launch_balance_bwd(const BalanceArgs& a, hipStream_t s) {
    by_experts(a.E, [&](auto lanes, auto vec) {
        const long tokens = 4 * (kWave / decltype(lanes)::value);  // of a workgroup at a time
        const long groups = (a.M + tokens - 1) / tokens;
        balance_bwd_kernel<decltype(lanes)::value, decltype(vec)::value>
            <<<(int)(groups < 2048 ? groups : 2048), 256, 0, s>>>(a);
    });
}

}  // namespace moe
