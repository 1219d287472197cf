// api_train.cpp -- the C ABI of the operators around the experts: matrix
// products grouped by expert, the gated activation between them and the norms
// around the block, with their gradients.  Arguments are checked before any
// HIP call, as in api.cpp.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/moe.h"
#include "launch.hpp"

#define MOE_API extern "C" __attribute__((visibility("default")))

namespace {

constexpr size_t kAlign = 256;
constexpr long kMaxRows = 1L << 28;     // sorted rows, slots
constexpr int kMaxWidth = 1 << 20;      // K, N
constexpr long kMaxThreads = 1L << 32;  // of a launch
constexpr long kMaxGather = 1L << 31;   // bytes of a gathered operand, of one expert's weights

bool misaligned(const void* p) { return p && ((uintptr_t)p & 15u); }
size_t round_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

// whether two buffers of these many bytes share any
bool overlap(const void* p, long np, const void* q, long nq) {
    const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
    return a < b + (uintptr_t)nq && b < a + (uintptr_t)np;
}

moe_status finish() { return hipGetLastError() == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// workspace == nullptr: reports the size.  Returns true when the call is done.
bool workspace_step(void* workspace, size_t* bytes, size_t need, moe_status* st) {
    if (need < kAlign) need = kAlign;  // never 0: a buffer sized from the query is not NULL
    if (!workspace) {
        *bytes = need;
        *st = MOE_OK;
        return true;
    }
    if ((uintptr_t)workspace & (kAlign - 1)) *st = MOE_ERR_INVALID_ARG;
    else if (*bytes < need) *st = MOE_ERR_WORKSPACE;
    else return false;
    return true;
}

// The size a product reports: the minimum exactly if it does not use it, so
// that a caller may pass any buffer then.
size_t product_size(size_t need) {
    return need == 0 ? 0 : need < 2 * kAlign ? 2 * kAlign : round_up(need);
}

// The checks that the three products share; fills g.  `flags`: the moe_rows
// bits the product knows.
moe_status grouped_setup(moe::GroupedArgs* g, const int32_t* offsets, const int32_t* sorted_ids,
                         int rows, int flags, int T, int topk, int R, int E, int K, int N) {
    if (rows & ~flags) return MOE_ERR_INVALID_ARG;
    if (T < 0 || topk < 1 || R < 0 || E < 1 || K < 1 || N < 1) return MOE_ERR_INVALID_ARG;
    if (rows && !sorted_ids && R > 0) return MOE_ERR_INVALID_ARG;
    const long slots = (long)T * topk;
    if (E > MOE_MAX_EXPERTS || topk > MOE_MAX_TOPK || R >= kMaxRows || slots >= kMaxRows ||
        K >= kMaxWidth || N >= kMaxWidth || (long)N * K * 2 >= kMaxGather)
        return MOE_ERR_UNSUPPORTED;
    // a launch of 64 x 64 output tiles, 256 threads each, rounded up to eight tiles
    const long wide = ((K > N ? K : N) + 63) / 64, most = kMaxThreads / 256 - 8;
    if (wide * (R / 64 + (long)E) >= most || (long)E * ((K + 63) / 64) * ((N + 63) / 64) >= most)
        return MOE_ERR_UNSUPPORTED;
    g->w = g->x = g->dy = nullptr;
    g->offsets = offsets;
    g->sorted = sorted_ids;
    g->how_x = g->how_dy = g->how_out = moe::kRowSorted;
    g->slots = (uint32_t)slots;
    g->magic = topk == 1 ? 0 : (uint32_t)(((1ull << 32) + topk - 1) / topk);
    g->T = T;
    g->R = R;
    g->E = E;
    g->K = K;
    g->N = N;
    g->out_f32 = g->accumulate = 0;
    g->splits = 1;
    g->out = nullptr;
    return MOE_OK;
}

// fwd (dx false) and dx
moe_status grouped_rows(bool dx, const void* in, const void* w, const int32_t* offsets,
                        const int32_t* sorted_ids, int rows, int T, int topk, int R, int E, int K,
                        int N, void* out, void* workspace, size_t* workspace_bytes, void* stream) {
    if (!workspace_bytes) return MOE_ERR_INVALID_ARG;
    moe::GroupedArgs g;
    // the size query has no pointers
    moe_status st = grouped_setup(&g, offsets, workspace ? sorted_ids : (const int32_t*)kAlign, rows,
                                  MOE_ROWS_GATHER | MOE_ROWS_SCATTER, T, topk, R, E, K, N);
    if (st != MOE_OK) return st;
    if ((rows & MOE_ROWS_GATHER) && (long)T * (dx ? N : K) * 2 >= kMaxGather)
        return MOE_ERR_UNSUPPORTED;
    const size_t need = dx ? moe::grouped_dx_workspace(g) : moe::grouped_fwd_workspace(g);
    if (workspace_step(workspace, workspace_bytes, product_size(need), &st)) return st;
    if (R == 0) return MOE_OK;
    // with T == 0 every row is padding, and a gathered / scattered operand has no rows
    if ((!in && !(T == 0 && (rows & MOE_ROWS_GATHER))) || !w || !offsets ||
        (!out && !(T == 0 && (rows & MOE_ROWS_SCATTER))))
        return MOE_ERR_INVALID_ARG;
    if (misaligned(in) || misaligned(w) || misaligned(offsets) || misaligned(sorted_ids) ||
        misaligned(out))
        return MOE_ERR_INVALID_ARG;
    // workgroups read all of an operand while others write
    const long slots = (long)T * topk, out_bytes = (rows & MOE_ROWS_SCATTER ? slots : R) * (dx ? K : N) * 2;
    if (overlap(out, out_bytes, in, (rows & MOE_ROWS_GATHER ? (long)T : R) * (dx ? N : K) * 2) ||
        overlap(out, out_bytes, w, (long)E * N * K * 2))
        return MOE_ERR_INVALID_ARG;
    const uint32_t how = rows & MOE_ROWS_GATHER ? moe::kRowToken : moe::kRowSorted;
    g.w = (const uint16_t*)w;
    (dx ? g.dy : g.x) = (const uint16_t*)in;
    (dx ? g.how_dy : g.how_x) = how;
    g.how_out = rows & MOE_ROWS_SCATTER ? moe::kRowSlot : moe::kRowSorted;
    g.out = out;
    (void)hipGetLastError();
    if (dx) moe::launch_grouped_dx(g, workspace, (hipStream_t)stream);
    else moe::launch_grouped_fwd(g, workspace, (hipStream_t)stream);
    return finish();
}

}  // namespace

MOE_API moe_status moe_grouped_gemm(const void* x, const void* w, const int32_t* expert_offsets,
                                    const int32_t* sorted_ids, int rows, int T, int topk, int R,
                                    int E, int K, int N, void* y, void* workspace,
                                    size_t* workspace_bytes, void* stream) {
    return grouped_rows(false, x, w, expert_offsets, sorted_ids, rows, T, topk, R, E, K, N, y,
                        workspace, workspace_bytes, stream);
}

MOE_API moe_status moe_grouped_gemm_dx(const void* dy, const void* w,
                                       const int32_t* expert_offsets, const int32_t* sorted_ids,
                                       int rows, int T, int topk, int R, int E, int K, int N,
                                       void* dx, void* workspace, size_t* workspace_bytes,
                                       void* stream) {
    return grouped_rows(true, dy, w, expert_offsets, sorted_ids, rows, T, topk, R, E, K, N, dx,
                        workspace, workspace_bytes, stream);
}

MOE_API moe_status moe_grouped_gemm_dw(const void* dy, const void* x,
                                       const int32_t* expert_offsets, const int32_t* sorted_ids,
                                       int rows, int T, int topk, int R, int E, int K, int N,
                                       int out, void* dw, void* workspace,
                                       size_t* workspace_bytes, void* stream) {
    if (!workspace_bytes) return MOE_ERR_INVALID_ARG;
    if (out < MOE_OUT_BF16 || out > MOE_OUT_FP32_ADD) return MOE_ERR_INVALID_ARG;
    moe::GroupedArgs g;
    // the size query has no pointers: rows that need sorted_ids are checked below
    moe_status st = grouped_setup(&g, expert_offsets, workspace ? sorted_ids : (const int32_t*)kAlign,
                                  rows, MOE_ROWS_GATHER | MOE_ROWS_GATHER_DY, T, topk, R, E, K, N);
    if (st != MOE_OK) return st;
    if (((rows & MOE_ROWS_GATHER) && (long)T * K * 2 >= kMaxGather) ||
        ((rows & MOE_ROWS_GATHER_DY) && (long)T * N * 2 >= kMaxGather))
        return MOE_ERR_UNSUPPORTED;
    g.out_f32 = out != MOE_OUT_BF16;
    g.accumulate = out == MOE_OUT_FP32_ADD;
    if (workspace_step(workspace, workspace_bytes, product_size(moe::grouped_dw_workspace(g)), &st))
        return st;
    if (R == 0 && g.accumulate) return MOE_OK;
    if (!expert_offsets || !dw) return MOE_ERR_INVALID_ARG;
    if (R > 0 && ((!dy && !(T == 0 && (rows & MOE_ROWS_GATHER_DY))) ||
                  (!x && !(T == 0 && (rows & MOE_ROWS_GATHER)))))
        return MOE_ERR_INVALID_ARG;
    if (misaligned(dy) || misaligned(x) || misaligned(expert_offsets) || misaligned(sorted_ids) ||
        misaligned(dw))
        return MOE_ERR_INVALID_ARG;
    const long dw_bytes = (long)E * N * K * (g.out_f32 ? 4 : 2);
    if (overlap(dw, dw_bytes, dy, (rows & MOE_ROWS_GATHER_DY ? (long)T : R) * N * 2) ||
        overlap(dw, dw_bytes, x, (rows & MOE_ROWS_GATHER ? (long)T : R) * K * 2))
        return MOE_ERR_INVALID_ARG;
    g.dy = (const uint16_t*)dy;
    g.x = (const uint16_t*)x;
    g.how_x = rows & MOE_ROWS_GATHER ? moe::kRowToken : moe::kRowSorted;
    g.how_dy = rows & MOE_ROWS_GATHER_DY ? moe::kRowToken : moe::kRowSorted;
    g.out = dw;
    (void)hipGetLastError();
    moe::launch_grouped_dw(g, workspace, (hipStream_t)stream);
    return finish();
}

MOE_API moe_status moe_grouped_plan(int op, int R, int E, int K, int N, moe_product_plan* plan) {
    if (!plan || op < MOE_PRODUCT_FWD || op > MOE_PRODUCT_DW) return MOE_ERR_INVALID_ARG;
    moe::GroupedArgs g;
    const moe_status st = grouped_setup(&g, nullptr, nullptr, 0, 0, 0, 1, R, E, K, N);
    if (st != MOE_OK) return st;
    const moe::GroupedPlan p = moe::grouped_plan(g, op);
    plan->kernel = p.kernel;
    plan->splits = p.splits;
    plan->workgroups = p.workgroups;
    plan->reserved = 0;
    size_t bytes = op == MOE_PRODUCT_DW   ? moe::grouped_dw_workspace(g)
                   : op == MOE_PRODUCT_DX ? moe::grouped_dx_workspace(g)
                                          : moe::grouped_fwd_workspace(g);
    bytes = product_size(bytes);
    plan->workspace_bytes = bytes < kAlign ? kAlign : bytes;
    return MOE_OK;
}

// ---- the gated activation ------------------------------------------------------

static moe_status gated_check(moe::GatedArgs* a, const void* g, const float* topk_weights,
                              const int32_t* sorted_ids, const int32_t* num_rows, int slots, int R,
                              int N) {
    if (slots < 0 || R < 0 || N < 1) return MOE_ERR_INVALID_ARG;
    if (R >= kMaxRows || slots >= kMaxRows || N >= kMaxWidth) return MOE_ERR_UNSUPPORTED;
    // a thread per 8 values, or a workgroup of 256 a row
    const long row = (N + 7) / 8;
    if ((long)R * (row > 256 ? row : 256) > kMaxThreads - 256) return MOE_ERR_UNSUPPORTED;
    // without sorted_ids row i is slot i
    if (topk_weights && !sorted_ids && slots < R) return MOE_ERR_INVALID_ARG;
    if (misaligned(g) || misaligned(topk_weights) || misaligned(sorted_ids) ||
        misaligned(num_rows))
        return MOE_ERR_INVALID_ARG;
    a->g = (const uint16_t*)g;
    a->da = nullptr;
    a->weights = topk_weights;
    a->sorted = sorted_ids;
    a->num_rows = num_rows;
    a->slots = (uint32_t)slots;
    a->R = R;
    a->N = N;
    a->out = nullptr;
    a->dweights = nullptr;
    return MOE_OK;
}

MOE_API moe_status moe_silu_mul(const void* g, const float* topk_weights,
                                const int32_t* sorted_ids, const int32_t* num_rows, int slots,
                                int R, int N, void* a, void* stream) {
    moe::GatedArgs args;
    const moe_status st = gated_check(&args, g, topk_weights, sorted_ids, num_rows, slots, R, N);
    if (st != MOE_OK) return st;
    if (R == 0) return MOE_OK;
    if (!g || !a || misaligned(a)) return MOE_ERR_INVALID_ARG;
    args.out = (uint16_t*)a;
    (void)hipGetLastError();
    moe::launch_silu_mul(args, (hipStream_t)stream);
    return finish();
}

MOE_API moe_status moe_silu_mul_bwd(const void* da, const void* g, const float* topk_weights,
                                    const int32_t* sorted_ids, const int32_t* num_rows, int slots,
                                    int R, int N, void* dg, float* dtopk_weights, void* stream) {
    moe::GatedArgs args;
    const moe_status st = gated_check(&args, g, topk_weights, sorted_ids, num_rows, slots, R, N);
    if (st != MOE_OK) return st;
    if (dtopk_weights && !topk_weights) return MOE_ERR_INVALID_ARG;
    if (R == 0) return MOE_OK;
    if (!da || !g || !dg || misaligned(da) || misaligned(dg) || misaligned(dtopk_weights))
        return MOE_ERR_INVALID_ARG;
    args.da = (const uint16_t*)da;
    args.out = (uint16_t*)dg;
    args.dweights = dtopk_weights;
    (void)hipGetLastError();
    moe::launch_silu_mul_bwd(args, (hipStream_t)stream);
    return finish();
}

// ---- the norms around a block ----------------------------------------------------

static moe_status norm_sizes(int h_dtype, int M, int K, int topk, int du_topk) {
    if (h_dtype != MOE_OUT_BF16 && h_dtype != MOE_OUT_FP32) return MOE_ERR_INVALID_ARG;
    if (M < 0 || K < 1 || topk < 1 || du_topk < 1) return MOE_ERR_INVALID_ARG;
    if (K >= kMaxWidth || topk > MOE_MAX_TOPK || du_topk > MOE_MAX_TOPK) return MOE_ERR_UNSUPPORTED;
    if ((long)M * topk >= kMaxRows || (long)M * du_topk >= kMaxRows) return MOE_ERR_UNSUPPORTED;
    if (M * 1024L >= kMaxThreads) return MOE_ERR_UNSUPPORTED;  // a workgroup a row
    return MOE_OK;
}

MOE_API moe_status moe_block_norm(const void* h, const void* o, const float* gate,
                                  const float* w_post, const float* w_pre, int h_dtype, int M,
                                  int K, int topk, float res_scale, float eps, void* h_out,
                                  void* u, float* rstd_post, float* rstd_pre, void* stream) {
    const moe_status st = norm_sizes(h_dtype, M, K, topk, 1);
    if (st != MOE_OK) return st;
    if (!(eps > 0.0f)) return MOE_ERR_INVALID_ARG;
    if (M == 0) return MOE_OK;
    if (!h || (!o && !w_pre)) return MOE_ERR_INVALID_ARG;
    if (!o && (gate || w_post || h_out)) return MOE_ERR_INVALID_ARG;
    if (o && !h_out) return MOE_ERR_INVALID_ARG;
    if (!w_pre != !u) return MOE_ERR_INVALID_ARG;
    if ((rstd_post && !w_post) || (rstd_pre && !w_pre)) return MOE_ERR_INVALID_ARG;
    if (misaligned(h) || misaligned(o) || misaligned(gate) || misaligned(w_post) ||
        misaligned(w_pre) || misaligned(h_out) || misaligned(u) || misaligned(rstd_post) ||
        misaligned(rstd_pre))
        return MOE_ERR_INVALID_ARG;
    moe::NormArgs a = {};
    a.h = h;
    a.o = (const uint16_t*)o;
    a.gate = gate;
    a.w_post = w_post;
    a.w_pre = w_pre;
    a.M = M;
    a.K = K;
    a.topk = topk;
    a.res_scale = res_scale;
    a.eps = eps;
    a.h_f32 = h_dtype == MOE_OUT_FP32;
    a.h_out = h_out;
    a.u = (uint16_t*)u;
    a.rstd_post = rstd_post;
    a.rstd_pre = rstd_pre;
    (void)hipGetLastError();
    moe::launch_block_norm(a, (hipStream_t)stream);
    return finish();
}

MOE_API moe_status moe_block_norm_bwd(const void* dh_out, const void* du, const void* h_out,
                                      const void* o, const float* gate, const float* w_post,
                                      const float* w_pre, const float* rstd_post,
                                      const float* rstd_pre, int h_dtype, int M, int K, int topk,
                                      int du_topk, float res_scale, void* dh, void* d_o,
                                      float* dgate, float* dw_post, float* dw_pre,
                                      void* workspace, size_t* workspace_bytes, void* stream) {
    if (!workspace_bytes) return MOE_ERR_INVALID_ARG;
    moe_status st = norm_sizes(h_dtype, M, K, topk, du_topk);
    if (st != MOE_OK) return st;
    // for both weights, whichever are asked for: the query has no pointers
    if (workspace_step(workspace, workspace_bytes,
                       round_up(moe::block_norm_bwd_workspace(M, K)), &st))
        return st;
    if (!w_post != !dw_post || !w_pre != !dw_pre) return MOE_ERR_INVALID_ARG;
    // without rows only the weights' gradients are written, and tensors of the
    // rows may be null
    if (M > 0) {
        if (!o && (gate || w_post || d_o || dgate)) return MOE_ERR_INVALID_ARG;
        if (!gate != !dgate) return MOE_ERR_INVALID_ARG;
        if (!dh || (!dh_out && !w_pre) || (!o && !w_pre)) return MOE_ERR_INVALID_ARG;
        if (!o != !d_o || !w_pre != !du) return MOE_ERR_INVALID_ARG;
        if (w_pre && (!h_out || !rstd_pre)) return MOE_ERR_INVALID_ARG;
        if (w_post && !rstd_post) return MOE_ERR_INVALID_ARG;
        // a row's inputs may be read again after its outputs are written
        if (dh == dh_out || dh == h_out || (d_o && (d_o == o || d_o == du)))
            return MOE_ERR_INVALID_ARG;
    }
    const void* all[] = {dh_out, du, h_out, o, gate, w_post, w_pre, rstd_post, rstd_pre,
                         dh, d_o, dgate, dw_post, dw_pre};
    for (const void* p : all)
        if (misaligned(p)) return MOE_ERR_INVALID_ARG;
    moe::NormArgs a = {};
    a.h = h_out;
    a.o = (const uint16_t*)o;
    a.du = (const uint16_t*)du;
    a.dh_out = dh_out;
    a.gate = gate;
    a.w_post = w_post;
    a.w_pre = w_pre;
    a.rstd_post_in = rstd_post;
    a.rstd_pre_in = rstd_pre;
    a.M = M;
    a.K = K;
    a.topk = topk;
    a.du_topk = du_topk;
    a.res_scale = res_scale;
    a.h_f32 = h_dtype == MOE_OUT_FP32;
    a.h_out = dh;
    a.u = (uint16_t*)d_o;
    a.dgate = dgate;
    a.dw_post = dw_post;
    a.dw_pre = dw_pre;
    (void)hipGetLastError();
    moe::launch_block_norm_bwd(a, (float*)workspace, (hipStream_t)stream);
    return finish();
}
