// balance.hip -- the balance loss of the router, the counts behind it, and the
// gradient of the logits.  V: the tokens that count (mask), n of them;
// p_t = softmax(l_t); c_e: slots of V's tokens that picked expert e:
//
//   f_e = c_e / (n k),   P_e = sum_{t in V} p_te / n,   loss = E sum_e f_e P_e
//   dl_te = dloss E / n  p_te (f_e - sum_i p_ti f_i),   zero rows outside V
//
// L <= 16 lanes share a token, and a lane C <= 4 groups of four experts (C > 1 with
// 16 lanes only), so a wave takes 64 / L tokens, and what a token's maximum and sums
// cost is shared by them.  Both passes are meant to be bound by HBM: the logits are
// read once, as 16 bytes a lane and group.  Sums are fp32 in a fixed order: a
// lane's tokens one after the other, then the lanes, the waves and the workgroups;
// counts are integers.  32768 tokens of 256 experts, a tenth masked, kernel times on
// average: forward 10.9-11.7 us (35 MB) and 4.7 to join the workgroups, backward 13.4-
// 15.0 us (67 MB, 4.5-5.0 TB/s); 15.6 and 14.9 us a call in a captured graph.  (With 64
// lanes a token, whose exchanges it then waits for, the forward took 1.5 times as
// long.)
#include "common.hpp"
#include "launch.hpp"

#include <type_traits>

namespace moe {

namespace {

constexpr int kSplit = 4;     // experts of a group
constexpr int kGroups = 256;  // workgroups of the forward at most: one a CU

// e^d for d <= 0 or NaN: 2^t with t = d log2 e, whose rounding is made good by the
// first term of its effect (2^t alone is off by |d| half steps)
__device__ __forceinline__ float exp_below(float d) {
    d = d < -150.0f ? -150.0f : d;
    const float t = d * 1.44269502f;
    const float rest = fmaf(d, 1.92596303e-8f, fmaf(d, 1.44269502f, -t));  // log2 e = 1.44269502 + 1.926e-8
    const float p = __builtin_amdgcn_exp2f(t);
    return fmaf(p, rest * 0.693147182f, p);
}

// experts of a token's lane: groups of four, 4 * L apart
template <int L, int C, bool VEC>
struct Token {
    f32x4_t v[C];

    __device__ static __forceinline__ int expert(int c) { return (c * L + lane_id() % L) * kSplit; }

    // -inf past the last expert
    __device__ __forceinline__ void load(const float* row, int E) {
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int e = expert(c);
#pragma unroll
            for (int i = 0; i < kSplit; ++i) v[c][i] = -__builtin_inff();
            if constexpr (VEC) {
                if (e < E) v[c] = *reinterpret_cast<const f32x4_t*>(row + e);
            } else {
#pragma unroll
                for (int i = 0; i < kSplit; ++i)
                    if (e + i < E) v[c][i] = row[e + i];
            }
        }
    }
    template <typename F>
    __device__ static __forceinline__ float reduce(float x, F f) {
        if constexpr (L > 1) x = f(x, __uint_as_float(xchg_u32<0>(__float_as_uint(x))));
        if constexpr (L > 2) x = f(x, __uint_as_float(xchg_u32<1>(__float_as_uint(x))));
        if constexpr (L > 4) x = f(x, __uint_as_float(xchg_u32<2>(__float_as_uint(x))));
        if constexpr (L > 8) x = f(x, __uint_as_float(xchg_u32<3>(__float_as_uint(x))));
        return x;
    }
    // the sum over the token's experts of g(group, place)
    template <typename G>
    __device__ static __forceinline__ float sum(G g) {
        float x = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) x += (g(c, 0) + g(c, 1)) + (g(c, 2) + g(c, 3));
        return reduce(x, [](float a, float b) { return a + b; });
    }
    // logits to probabilities; zeros where all are -inf (a NaN makes all of them NaN)
    __device__ __forceinline__ void softmax() {
        float m = -__builtin_inff();
#pragma unroll
        for (int c = 0; c < C; ++c) m = fmaxf(fmaxf(fmaxf(v[c][0], v[c][1]), fmaxf(v[c][2], v[c][3])), m);
        m = reduce(m, [](float a, float b) { return fmaxf(a, b); });
        const float base = m == -__builtin_inff() ? 0.0f : m;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < kSplit; ++i) v[c][i] = exp_below(v[c][i] - base);
        const float s = sum([&](int c, int i) { return v[c][i]; });
        float r = __builtin_amdgcn_rcpf(s);
        r = s == 0.0f ? 0.0f : fmaf(fmaf(-s, r, 1.0f), r, r);  // within half a step
#pragma unroll
        for (int c = 0; c < C; ++c) v[c] *= r;
    }
};

// counts and probs of expert e from the sums of all tokens; its share of the loss / E
__device__ __forceinline__ float balance_expert(const BalanceArgs& a, int e, float psum, int count, int n) {
    const float P = n > 0 ? psum / (float)n : 0.0f;
    a.counts[e] = count;
    a.probs[e] = P;
    return n > 0 ? (float)count / ((float)n * (float)a.topk) * P : 0.0f;
}

// Sums of many workgroups, in the workspace: [groups][E] of p, [groups][E] of
// counts, [groups] of tokens, a share of the loss for every 32 experts, and how many
// of these are written.
constexpr int kJoinExperts = 32, kJoinSlices = 32;
struct BalanceSums {
    float* p;
    int *counts, *tokens;
    float* shares;
    uint32_t* done;
};
BalanceSums balance_sums(void* workspace, int groups, int E) {
    BalanceSums s;
    s.p = (float*)workspace;
    s.counts = (int*)(s.p + (size_t)groups * E);
    s.tokens = s.counts + (size_t)groups * E;
    s.shares = (float*)(s.tokens + groups);
    s.done = (uint32_t*)(s.shares + 256 / kJoinExperts);
    return s;
}
size_t balance_sums_bytes(int groups, int E) { return ((size_t)groups * (2 * E + 1) + 256 / kJoinExperts + 1) * 4; }

// A workgroup takes the tokens [b, b + 1) * per; with more than one of them each
// leaves its sums in the workspace.  A wave loads two rounds of tokens and their
// masks at a time, and a thread its first slot's id before.
constexpr int kBalanceThreads = 512, kBalanceWaves = kBalanceThreads / kWave, kRounds = 2;

template <int L, int C, bool VEC>
__global__ __launch_bounds__(kBalanceThreads) void balance_kernel(BalanceArgs a, int per, BalanceSums to) {
    __shared__ float sums[kBalanceWaves][256];
    __shared__ int hist[256];
    __shared__ int seen[kBalanceWaves];
    __shared__ float part[4];
    constexpr int TW = kWave / L, kStep = kBalanceWaves * TW;  // tokens a wave, a round
    const int tid = (int)threadIdx.x, lane = lane_id(), wave = tid / kWave;
    const int first = (int)blockIdx.x * per, last = min(first + per, a.M);
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    const uint32_t s0 = (uint32_t)first * (uint32_t)a.topk + (uint32_t)tid, s1 = (uint32_t)last * (uint32_t)a.topk;
    uint32_t pick = 0, valid = 0;
    if (s0 < s1) {
        pick = (uint32_t)a.ids[s0];
        valid = a.mask ? a.mask[s0 / (uint32_t)a.topk] : 1u;
    }
    f32x4_t acc[C];
#pragma unroll
    for (int c = 0; c < C; ++c) acc[c] = f32x4_t{0, 0, 0, 0};
    int tokens = 0;
    for (int t0 = first + wave * TW; t0 < last; t0 += kRounds * kStep) {
        Token<L, C, VEC> p[kRounds];
        uint32_t in[kRounds];  // masks as loaded: a comparison would wait for them
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            const int t = t0 + r * kStep + lane / L;
            in[r] = 0;
#pragma unroll
            for (int c = 0; c < C; ++c) p[r].v[c] = f32x4_t{0, 0, 0, 0};
            if (t < last) {
                in[r] = a.mask ? a.mask[t] : 1u;
                p[r].load(a.logits + (size_t)t * a.E, a.E);
            }
        }
#pragma unroll
        for (int r = 0; r < kRounds; ++r) {
            p[r].softmax();
            tokens += in[r] != 0 && lane % L == 0;
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (in[r] != 0) acc[c] += p[r].v[c];
        }
    }
    for (uint32_t s = s0; s < s1;) {
        if (valid != 0 && pick < (uint32_t)a.E) atomicAdd(&hist[pick], 1);
        s += kBalanceThreads;
        if (s < s1) {
            pick = (uint32_t)a.ids[s];
            valid = a.mask ? a.mask[s / (uint32_t)a.topk] : 1u;
        }
    }
    // lanes with the same experts, then the waves
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < kSplit; ++i) {
            float v = acc[c][i];
#pragma unroll
            for (int d = L; d < kWave; d *= 2) v += __shfl_xor(v, d);
            if (lane < L) sums[wave][Token<L, C, VEC>::expert(c) + i] = v;
        }
#pragma unroll
    for (int d = 1; d < kWave; d *= 2) tokens += __shfl_xor(tokens, d);
    if (lane == 0) seen[wave] = tokens;
    __syncthreads();
    if (tid >= 256) return;
    float psum = 0.0f;
    int n = 0;
#pragma unroll
    for (int w = 0; w < kBalanceWaves; ++w) {
        if (tid < L * C * kSplit) psum += sums[w][tid];
        n += seen[w];
    }
    if (gridDim.x > 1) {
        if (tid < a.E) {
            to.p[(size_t)blockIdx.x * a.E + tid] = psum;
            to.counts[(size_t)blockIdx.x * a.E + tid] = hist[tid];
        }
        if (tid == 0) to.tokens[blockIdx.x] = n;
        if (tid == 0 && blockIdx.x == 0) *to.done = 0;  // for the next launch
        return;
    }
    const float term = wave_sum_f32(tid < a.E ? balance_expert(a, tid, psum, hist[tid], n) : 0.0f);
    if (lane == 0) part[wave] = term;
    __syncthreads();
    if (tid == 0) {
        a.tokens[0] = n;
        a.loss[0] = (float)a.E * ((part[0] + part[1]) + (part[2] + part[3]));
    }
}

// The workgroups' sums, 32 experts a workgroup and 32 threads an expert, in an order
// of their own.  The workgroup that is done last adds up the shares of the loss, in the
// order of the experts whichever it is.  (One workgroup for all of 256 experts
// is bound by what a CU can load: 7.0 us of 256 groups' sums.)
__global__ __launch_bounds__(kJoinExperts* kJoinSlices) void balance_join_kernel(BalanceArgs a, int groups,
                                                                                 BalanceSums from) {
    __shared__ float ps[kJoinSlices][kJoinExperts];
    __shared__ int cs[kJoinSlices][kJoinExperts], ts[4];
    const int tid = (int)threadIdx.x, i = tid % kJoinExperts, q = tid / kJoinExperts;
    const int e = (int)blockIdx.x * kJoinExperts + i;
    float p = 0.0f;
    int c = 0;
    if (e < a.E) {
#pragma unroll 8
        for (int g = q; g < groups; g += kJoinSlices) {
            p += from.p[(size_t)g * a.E + e];
            c += from.counts[(size_t)g * a.E + e];
        }
    }
    ps[q][i] = p;
    cs[q][i] = c;
    if (tid < 256) {
        int n = tid < groups ? from.tokens[tid] : 0;
#pragma unroll
        for (int d = 1; d < kWave; d *= 2) n += __shfl_xor(n, d);
        if (lane_id() == 0) ts[tid / kWave] = n;
    }
    __syncthreads();
    if (tid >= kWave) return;
    const int n = (ts[0] + ts[1]) + (ts[2] + ts[3]);
    float term = 0.0f;
    if (tid < kJoinExperts && e < a.E) {
        p = ps[0][i];
        c = cs[0][i];
#pragma unroll
        for (int s = 1; s < kJoinSlices; ++s) {
            p += ps[s][i];
            c += cs[s][i];
        }
        term = balance_expert(a, e, p, c, n);
    }
    term = wave_sum_f32(term);
    if (tid != 0) return;
    if (blockIdx.x == 0) a.tokens[0] = n;
    __hip_atomic_store(from.shares + blockIdx.x, term, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    const uint32_t before = __hip_atomic_fetch_add(from.done, 1u, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT);
    if (before + 1 < gridDim.x) return;
    float loss = 0.0f;
    for (int b = 0; b < (int)gridDim.x; ++b)
        loss += __hip_atomic_load(from.shares + b, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    a.loss[0] = (float)a.E * loss;
}

// A wave's next tokens are loaded before the present ones are worked on, and results
// do not stay in the L2 (32768 x 256: 12.4 us, 15.5 in ordinary stores; 2048
// workgroups, which go around once, 16.7).  (The logits of a token that does not
// count may be anything: its gradient is written as zeros whatever was computed.)
constexpr int kBwdGroups = 1024;  // workgroups at most

template <int L, int C, bool VEC>
__global__ __launch_bounds__(256) void balance_bwd_kernel(BalanceArgs a) {
    typedef Token<L, C, VEC> token_t;
    constexpr int TW = kWave / L;
    const long stride = (long)gridDim.x * 4 * TW;
    token_t next;
    uint32_t mask = 1;
    auto load = [&](long t) {
        if (t < a.M) {
            next.load(a.logits + (size_t)t * a.E, a.E);
            if (a.mask) mask = a.mask[t];
        }
    };
#pragma unroll
    for (int c = 0; c < C; ++c) next.v[c] = f32x4_t{0, 0, 0, 0};
    long t0 = ((long)blockIdx.x * 4 + threadIdx.x / kWave) * TW;
    load(t0 + lane_id() / L);
    const int n = a.tokens[0];
    const float inv = n > 0 ? 1.0f / (float)n : 0.0f, share = inv / (float)a.topk;
    float f[C][kSplit];
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int i = 0; i < kSplit; ++i) {
            const int e = token_t::expert(c) + i;
            f[c][i] = e < a.E ? (float)a.counts[e] * share : 0.0f;
        }
    const float up = a.dloss[0] * (float)a.E * inv;
    for (; t0 < a.M; t0 += stride) {
        const long t = t0 + lane_id() / L;
        const bool in = t < a.M, counts = in && n > 0 && mask != 0;
        token_t p = next;
        load(t + stride);
        p.softmax();
        const float dot = token_t::sum([&](int c, int i) { return p.v[c][i] * f[c][i]; });
#pragma unroll
        for (int c = 0; c < C; ++c) {
            f32x4_t d;
#pragma unroll
            for (int i = 0; i < kSplit; ++i) d[i] = counts ? up * p.v[c][i] * (f[c][i] - dot) : 0.0f;
            if (!in) continue;
            const int e = token_t::expert(c);
            float* o = a.dlogits + (size_t)t * a.E + e;
            if constexpr (VEC) {
                if (e < a.E) __builtin_nontemporal_store(d, reinterpret_cast<f32x4_t*>(o));
            } else {
#pragma unroll
                for (int i = 0; i < kSplit; ++i)
                    if (e + i < a.E) o[i] = d[i];
            }
        }
    }
}

// calls f(lanes a token, groups a lane, whether rows are whole vectors)
template <typename F>
void by_experts(int E, F f) {
    auto vec = [&](auto lanes, auto groups) {
        if (E % kSplit == 0) f(lanes, groups, std::true_type{});
        else f(lanes, groups, std::false_type{});
    };
    const std::integral_constant<int, 1> one;
    const std::integral_constant<int, 16> most;
    if (E <= 4) vec(one, one);
    else if (E <= 8) vec(std::integral_constant<int, 2>{}, one);
    else if (E <= 16) vec(std::integral_constant<int, 4>{}, one);
    else if (E <= 32) vec(std::integral_constant<int, 8>{}, one);
    else if (E <= 64) vec(most, one);
    else if (E <= 128) vec(most, std::integral_constant<int, 2>{});
    else if (E <= 192) vec(most, std::integral_constant<int, 3>{});
    else vec(most, std::integral_constant<int, 4>{});
}

// Tokens a workgroup.  All of them while a second launch would cost more than its
// share of the work (512 tokens of 8 experts: 12 us a call, 16 in two launches);
// then a load of every thread or more, and a workgroup a CU at most.
int balance_per(int M, int E) {
    if ((long)M * E <= 4 * kBalanceThreads * kSplit) return M;
    const int per = (kBalanceThreads * kSplit + E - 1) / E, share = (M + kGroups - 1) / kGroups;
    return per > share ? per : share;
}
int balance_groups(int M, int E) { return M == 0 ? 1 : (M + balance_per(M, E) - 1) / balance_per(M, E); }

}  // namespace

size_t balance_workspace(int M, int E) {
    const int groups = balance_groups(M, E);
    return groups > 1 ? balance_sums_bytes(groups, E) : 0;
}

void launch_balance(const BalanceArgs& a, void* workspace, hipStream_t s) {
    const int groups = balance_groups(a.M, a.E), per = balance_per(a.M, a.E);
    const BalanceSums sums = balance_sums(workspace, groups, a.E);
    by_experts(a.E, [&](auto lanes, auto of_lane, auto vec) {
        balance_kernel<decltype(lanes)::value, decltype(of_lane)::value, decltype(vec)::value>
            <<<groups, kBalanceThreads, 0, s>>>(a, per, sums);
    });
    if (groups > 1)
        balance_join_kernel<<<(a.E + kJoinExperts - 1) / kJoinExperts, kJoinExperts * kJoinSlices, 0, s>>>(a, groups,
                                                                                                          sums);
}

void launch_balance_bwd(const BalanceArgs& a, hipStream_t s) {
    by_experts(a.E, [&](auto lanes, auto of_lane, auto vec) {
        const long tokens = 4 * (kWave / decltype(lanes)::value);  // of a workgroup at a time
        const long groups = (a.M + tokens - 1) / tokens;
        balance_bwd_kernel<decltype(lanes)::value, decltype(of_lane)::value, decltype(vec)::value>
            <<<(int)(groups < kBwdGroups ? groups : kBwdGroups), 256, 0, s>>>(a);
    });
}

}  // namespace moe
