// api_ckpt.cpp -- the C ABI of the activations kept in 8 bits.  Arguments are
// checked before any HIP call, as in api.cpp.
#include "api_checks.hpp"
#include "ckpt_sizes.hpp"
#include "launch.hpp"

using namespace moe;

namespace {

// a launch has a thread per 8 columns, blocks of 32 columns whole
bool too_many(long R, long W) { return R * (ckpt_blocks((int)W) * 4L) > kMaxThreads - 256; }

moe_status rows_sizes(int R, int W) {
    if (R < 0 || W < 1) return MOE_ERR_INVALID_ARG;
    if (R >= kMaxRows || W >= kMaxWidth || too_many(R, W)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

}  // namespace

MOE_API moe_status moe_ckpt_rows(const void* x, int R, int W, int8_t* codes, uint8_t* scales,
                                 void* stream) {
    const moe_status st = rows_sizes(R, W);
    if (st != MOE_OK) return st;
    if (R == 0) return MOE_OK;
    if (!x || !codes || !scales || misaligned(x) || misaligned(codes) || misaligned(scales))
        return MOE_ERR_INVALID_ARG;
    const long n = (long)R * W;
    if (overlaps<2, 1>({{codes, n}, {scales, (long)R * ckpt_blocks(W)}}, {{x, 2 * n}}))
        return MOE_ERR_INVALID_ARG;
    (void)hipGetLastError();
    launch_ckpt_rows((const uint16_t*)x, R, W, codes, scales, (hipStream_t)stream);
    return finish();
}

MOE_API moe_status moe_ckpt_restore(const int8_t* codes, const uint8_t* scales, int R, int W, void* x,
                                    void* stream) {
    const moe_status st = rows_sizes(R, W);
    if (st != MOE_OK) return st;
    if (R == 0) return MOE_OK;
    if (!x || !codes || !scales || misaligned(x) || misaligned(codes) || misaligned(scales))
        return MOE_ERR_INVALID_ARG;
    const long n = (long)R * W;
    if (overlaps<1, 2>({{x, 2 * n}}, {{codes, n}, {scales, (long)R * ckpt_blocks(W)}}))
        return MOE_ERR_INVALID_ARG;
    (void)hipGetLastError();
    launch_ckpt_restore(codes, scales, R, W, (uint16_t*)x, (hipStream_t)stream);
    return finish();
}

// ---- the gated activation -------------------------------------------------------

static moe_status gated_check(GatedCkptArgs* a, const float* topk_weights, const int32_t* sorted_ids,
                              const int32_t* num_rows, int slots, int R, int N) {
    if (slots < 0 || R < 0 || N < 1) return MOE_ERR_INVALID_ARG;
    if (R >= kMaxRows || slots >= kMaxRows || N >= kMaxWidth || too_many(R, N) ||
        R * 256L > kMaxThreads - 256)
        return MOE_ERR_UNSUPPORTED;
    // without sorted_ids row i is slot i
    if (topk_weights && !sorted_ids && slots < R) return MOE_ERR_INVALID_ARG;
    if (misaligned(topk_weights) || misaligned(sorted_ids) || misaligned(num_rows))
        return MOE_ERR_INVALID_ARG;
    *a = {};
    a->weights = topk_weights;
    a->sorted = sorted_ids;
    a->num_rows = num_rows;
    a->slots = (uint32_t)slots;
    a->R = R;
    a->N = N;
    return MOE_OK;
}

MOE_API moe_status moe_silu_mul_ckpt(const void* g, const float* topk_weights,
                                     const int32_t* sorted_ids, const int32_t* num_rows, int slots,
                                     int R, int N, void* a, int8_t* codes, uint8_t* scales,
                                     void* stream) {
    GatedCkptArgs args;
    const moe_status st = gated_check(&args, topk_weights, sorted_ids, num_rows, slots, R, N);
    if (st != MOE_OK) return st;
    if (R == 0) return MOE_OK;
    if (!g || !a || !codes || !scales || misaligned(g) || misaligned(a) || misaligned(codes) ||
        misaligned(scales))
        return MOE_ERR_INVALID_ARG;
    const long n = (long)R * N, held = 2L * R * ckpt_blocks(N);
    if (overlaps<3, 4>({{a, 2 * n}, {codes, 2 * n}, {scales, held}},
                       {{g, 4 * n}, {topk_weights, 4L * slots}, {sorted_ids, 4L * R}, {num_rows, 4}}))
        return MOE_ERR_INVALID_ARG;
    args.g = (const uint16_t*)g;
    args.out = (uint16_t*)a;
    args.codes_out = codes;
    args.scales_out = scales;
    (void)hipGetLastError();
    launch_silu_mul_ckpt(args, (hipStream_t)stream);
    return finish();
}

MOE_API moe_status moe_silu_mul_bwd_ckpt(const void* da, const int8_t* codes, const uint8_t* scales,
                                         const float* topk_weights, const int32_t* sorted_ids,
                                         const int32_t* num_rows, int slots, int R, int N, void* dg,
                                         float* dtopk_weights, void* a, void* stream) {
    GatedCkptArgs args;
    const moe_status st = gated_check(&args, topk_weights, sorted_ids, num_rows, slots, R, N);
    if (st != MOE_OK) return st;
    if (dtopk_weights && !topk_weights) return MOE_ERR_INVALID_ARG;
    if (R == 0) return MOE_OK;
    if (!da || !codes || !scales || !dg || misaligned(da) || misaligned(codes) || misaligned(scales) ||
        misaligned(dg) || misaligned(dtopk_weights) || misaligned(a))
        return MOE_ERR_INVALID_ARG;
    const long n = (long)R * N, held = 2L * R * ckpt_blocks(N);
    if (overlaps<3, 6>({{dg, 4 * n}, {a, 2 * n}, {dtopk_weights, 4L * slots}},
                       {{da, 2 * n}, {codes, 2 * n}, {scales, held}, {topk_weights, 4L * slots},
                        {sorted_ids, 4L * R}, {num_rows, 4}}))
        return MOE_ERR_INVALID_ARG;
    args.da = (const uint16_t*)da;
    args.codes = codes;
    args.scales = scales;
    args.out = (uint16_t*)dg;
    args.dweights = dtopk_weights;
    args.again = (uint16_t*)a;
    (void)hipGetLastError();
    launch_silu_mul_bwd_ckpt(args, (hipStream_t)stream);
    return finish();
}
