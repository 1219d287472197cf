// api_router.cpp -- the C ABI of the router's balance loss and gradients.
// Arguments are checked before any HIP call, as in api.cpp.
#include "api_checks.hpp"
#include "launch.hpp"

using namespace moe;

namespace {

moe_status router_sizes(int M, int E, int topk) {
    if (M < 0 || E < 1 || topk < 1 || topk > E) return MOE_ERR_INVALID_ARG;
    if (E > MOE_MAX_EXPERTS || topk > MOE_MAX_TOPK || (long)M * topk >= kMaxRows)
        return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

}  // namespace

MOE_API moe_status moe_balance(const float* logits, const int32_t* topk_ids, const uint8_t* token_mask,
                               int M, int E, int topk, float* loss, int32_t* counts, int32_t* tokens,
                               float* probs, void* workspace, size_t* workspace_bytes, void* stream) {
    if (!workspace_bytes) return MOE_ERR_INVALID_ARG;
    moe_status st = router_sizes(M, E, topk);
    if (st != MOE_OK) return st;
    if (workspace_step(workspace, workspace_bytes, used_size(balance_workspace(M, E)), &st)) return st;
    if (!loss || !counts || !tokens || !probs || (M > 0 && (!logits || !topk_ids)))
        return MOE_ERR_INVALID_ARG;
    const void* all[] = {logits, topk_ids, token_mask, loss, counts, tokens, probs};
    for (const void* p : all)
        if (misaligned(p)) return MOE_ERR_INVALID_ARG;
    if (overlaps<4, 3>({{loss, 4}, {counts, 4L * E}, {tokens, 4}, {probs, 4L * E}},
                       {{logits, 4L * M * E}, {topk_ids, 4L * M * topk}, {token_mask, M}}))
        return MOE_ERR_INVALID_ARG;
    BalanceArgs a = {};
    a.logits = logits;
    a.ids = topk_ids;
    a.mask = token_mask;
    a.M = M;
    a.E = E;
    a.topk = topk;
    a.loss = loss;
    a.probs = probs;
    a.counts = counts;
    a.tokens = tokens;
    (void)hipGetLastError();
    launch_balance(a, workspace, (hipStream_t)stream);
    return finish();
}

MOE_API moe_status moe_balance_bwd(const float* dloss, const float* logits, const int32_t* counts,
                                   const int32_t* tokens, const uint8_t* token_mask, int M, int E,
                                   int topk, float* dlogits, void* stream) {
    const moe_status st = router_sizes(M, E, topk);
    if (st != MOE_OK) return st;
    if (M == 0) return MOE_OK;
    if (!dloss || !logits || !counts || !tokens || !dlogits) return MOE_ERR_INVALID_ARG;
    const void* all[] = {dloss, logits, counts, tokens, token_mask, dlogits};
    for (const void* p : all)
        if (misaligned(p)) return MOE_ERR_INVALID_ARG;
    if (overlaps<1, 5>({{dlogits, 4L * M * E}},
                       {{dloss, 4}, {logits, 4L * M * E}, {counts, 4L * E}, {tokens, 4}, {token_mask, M}}))
        return MOE_ERR_INVALID_ARG;
    BalanceArgs a = {};
    a.logits = logits;
    a.mask = token_mask;
    a.M = M;
    a.E = E;
    a.topk = topk;
    a.counts = const_cast<int32_t*>(counts);
    a.tokens = const_cast<int32_t*>(tokens);
    a.dloss = dloss;
    a.dlogits = dlogits;
    (void)hipGetLastError();
    launch_balance_bwd(a, (hipStream_t)stream);
    return finish();
}

MOE_API moe_status moe_topk_bwd(const void* x, const void* w_router, const int32_t* topk_ids,
                                const float* topk_weights, const float* dtopk_weights,
                                const float* dlogits, const void* dx_rows, int rows, int M, int K,
                                int E, int topk, void* dx, float* dw, float* dbias, void* workspace,
                                size_t* workspace_bytes, void* stream) {
    if (!workspace_bytes) return MOE_ERR_INVALID_ARG;
    moe_status st = router_sizes(M, E, topk);
    if (st != MOE_OK) return st;
    if (K < 1 || rows < 0) return MOE_ERR_INVALID_ARG;
    if (K >= kMaxWidth || rows > MOE_MAX_TOPK || (long)M * rows >= kMaxRows ||
        router_bwd_workgroups(M, K, E) * 256 >= kMaxThreads)
        return MOE_ERR_UNSUPPORTED;
    if (workspace_step(workspace, workspace_bytes, used_size(router_bwd_workspace(M, K, E)), &st)) return st;
    if (!dw) return MOE_ERR_INVALID_ARG;
    if (M > 0) {
        if (!x || !w_router || !dx || !dx_rows != !rows) return MOE_ERR_INVALID_ARG;
        if (!topk_ids != !topk_weights || !topk_ids != !dtopk_weights || (!topk_ids && !dlogits))
            return MOE_ERR_INVALID_ARG;
    }
    const void* all[] = {x,  w_router, topk_ids, topk_weights, dtopk_weights, dlogits, dx_rows,
                         dx, dw,       dbias};
    for (const void* p : all)
        if (misaligned(p)) return MOE_ERR_INVALID_ARG;
    const long n = 2L * M * K, nk = 4L * M * topk;
    if (overlaps<3, 7>({{dx, n}, {dw, 4L * E * K}, {dbias, 4L * E}},
                       {{x, n}, {w_router, 2L * E * K}, {topk_ids, nk}, {topk_weights, nk},
                        {dtopk_weights, nk}, {dlogits, 4L * M * E}, {dx_rows, n * rows}}))
        return MOE_ERR_INVALID_ARG;
    RouterBwdArgs a = {};
    a.x = (const uint16_t*)x;
    a.w = (const uint16_t*)w_router;
    a.ids = topk_ids;
    a.weights = topk_weights;
    a.dweights = dtopk_weights;
    a.dlogits = dlogits;
    a.dx_rows = (const uint16_t*)dx_rows;
    a.rows = rows;
    a.M = M;
    a.K = K;
    a.E = E;
    a.topk = topk;
    a.dx = (uint16_t*)dx;
    a.dw = dw;
    a.dbias = dbias;
    (void)hipGetLastError();
    launch_router_bwd(a, workspace, (hipStream_t)stream);
    return finish();
}
