// abi_ops.cu -- extern "C" entry points of the operators around the linears
// (declared in include/sharq.h).  Arguments are validated here, on the host,
// before anything is enqueued; the kernels live in norm.cu, route.cu and
// int8.cu.
#include "../../include/sharq.h"
#include "ops_internal.h"
#include "sharq_internal.h"

#include <cmath>

namespace {

constexpr int64_t kMaxInt = 2147483647;
constexpr int64_t kMaxRows8 = (int64_t)1 << 30;     // rows of an 8-bit operand: tile starts stay in int32

bool aligned(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

sharq_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return SHARQ_OK;
    cudaGetLastError();                       // reported here: not left for the caller's next check
    if (e == cudaErrorNotSupported) return SHARQ_ERR_UNSUPPORTED;
    return SHARQ_ERR_CUDA;
}

// A row stride in elements of `size` bytes over rows of K elements, every
// row start 16-byte aligned.
bool valid_ld(int64_t ld, int K, int64_t rows, int size) {
    return (rows <= 1 || ld >= K) && ld >= 0 && ld <= ((int64_t)1 << 40) && ld * size % 16 == 0;
}

bool valid_routing(const sharq_routing* r) {
    return r && r->T >= 0 && r->k >= 1 && r->E >= 1 && r->E <= 512 && r->T <= kMaxInt / r->k;
}

bool valid_norm_extent(int64_t M, int K) { return M >= 0 && M <= kMaxInt && K >= 8 && K <= 32768 && K % 8 == 0; }

bool valid_eps(float eps) { return eps >= 0.0f && eps < 1e30f; }

bool valid_rows8(const int8_t* codes, const float* scales, int64_t rows) {
    return rows == 0 || (codes && scales && aligned(codes, 16) && aligned(scales, 4));
}

// Rows of X quantised to 8 bits, after an RMSNorm when gamma is given.
sharq_status quantize_rows(const void* X, const void* gamma, float eps, int8_t* codes, float* scales,
                           int64_t M, int K, void* stream) {
    if (!valid_norm_extent(M, K) || !valid_eps(eps) || !valid_rows8(codes, scales, M))
        return SHARQ_ERR_INVALID_ARG;
    if ((M > 0 && !X) || !aligned(X, 16) || !aligned(gamma, 16)) return SHARQ_ERR_INVALID_ARG;
    sharq::NormLaunch p{};
    p.x = X; p.ldx = K; p.M = M; p.K = K; p.group_rows = M; p.alpha = 1.0f;
    p.gamma = gamma; p.norm = gamma ? SHARQ_NORM_RMS : SHARQ_NORM_NONE; p.eps = eps;
    p.codes = codes; p.row_scale = scales;
    return cuda_status(sharq::launch_residual_norm(p, static_cast<cudaStream_t>(stream), sharq::device_sm_count()));
}

}  // namespace

extern "C" {

sharq_status sharq_moe_dispatch(const sharq_routing* r, void* stream) {
    if (!valid_routing(r) || !r->offsets || !aligned(r->offsets, 4)) return SHARQ_ERR_INVALID_ARG;
    if (r->T > 0 && (!r->ids || !r->row_index || !r->position)) return SHARQ_ERR_INVALID_ARG;
    if (!aligned(r->ids, 4) || !aligned(r->row_index, 4) || !aligned(r->position, 4)) return SHARQ_ERR_INVALID_ARG;
    sharq::DispatchLaunch p{r->ids, r->row_index, r->offsets, r->position, r->T * r->k, r->E, r->k};
    return cuda_status(sharq::launch_dispatch(p, static_cast<cudaStream_t>(stream)));
}

sharq_status sharq_moe_route(const void* logits, int64_t ld, int logits_fp32, const float* bias,
                             const sharq_route_options* opt, const sharq_routing* out, void* stream) {
    if (!opt || !valid_routing(out) || out->k > 32) return SHARQ_ERR_INVALID_ARG;
    if (opt->score != SHARQ_SCORE_SOFTMAX && opt->score != SHARQ_SCORE_SIGMOID) return SHARQ_ERR_INVALID_ARG;
    if (opt->group_score != SHARQ_GROUP_MAX && opt->group_score != SHARQ_GROUP_TOP2) return SHARQ_ERR_INVALID_ARG;
    if (opt->groups < 1 || opt->groups > 32 || out->E % opt->groups != 0) return SHARQ_ERR_INVALID_ARG;
    if (opt->topk_groups < 1 || opt->topk_groups > opt->groups ||
        out->k > out->E / opt->groups * opt->topk_groups)
        return SHARQ_ERR_INVALID_ARG;
    if (!std::isfinite(opt->scale)) return SHARQ_ERR_INVALID_ARG;
    if (out->T > 0 && (!logits || !out->ids || !out->weights)) return SHARQ_ERR_INVALID_ARG;
    if (!aligned(logits, logits_fp32 ? 4 : 2) || !aligned(bias, 4) || !aligned(out->ids, 4) ||
        !aligned(out->weights, 4) || (out->T > 1 && ld < out->E) || ld < 0 || ld > ((int64_t)1 << 40))
        return SHARQ_ERR_INVALID_ARG;
    const bool order = out->row_index || out->offsets || out->position;
    if (order && (!out->offsets || (out->T > 0 && (!out->row_index || !out->position)) ||
                  !aligned(out->row_index, 4) || !aligned(out->offsets, 4) || !aligned(out->position, 4)))
        return SHARQ_ERR_INVALID_ARG;
    sharq::RouteLaunch p{};
    p.logits = logits; p.ld = ld; p.fp32 = logits_fp32 ? 1 : 0; p.bias = bias;
    p.ids = out->ids; p.weights = out->weights; p.T = out->T; p.E = out->E; p.k = out->k;
    p.sigmoid = opt->score == SHARQ_SCORE_SIGMOID; p.groups = opt->groups; p.topk_groups = opt->topk_groups;
    p.group_top2 = opt->group_score == SHARQ_GROUP_TOP2; p.renormalize = opt->renormalize ? 1 : 0;
    p.scale = opt->scale;
    const sharq::DispatchLaunch d{out->ids, out->row_index, out->offsets, out->position, out->T * out->k, out->E, out->k};
    return cuda_status(sharq::launch_route(p, order ? &d : nullptr, static_cast<cudaStream_t>(stream),
                                           sharq::device_sm_count()));
}

sharq_status sharq_moe_combine(const void* Y, int y_is_fp32, int64_t rows, int N, const int32_t* position,
                               const float* weights, int64_t T, int k, const void* residual, void* out,
                               int out_is_fp32, void* stream) {
    if (T < 0 || T > kMaxInt || rows < 0 || k < 1 || N < 8 || N % 8 != 0 || N > (1 << 24)) return SHARQ_ERR_INVALID_ARG;
    if (T > 0 && (!position || !weights || !out)) return SHARQ_ERR_INVALID_ARG;
    if (rows > 0 && !Y) return SHARQ_ERR_INVALID_ARG;
    if (!aligned(Y, 16) || !aligned(residual, 16) || !aligned(out, 16) || !aligned(position, 4) ||
        !aligned(weights, 4))
        return SHARQ_ERR_INVALID_ARG;
    sharq::CombineLaunch p{Y, position, weights, residual, out, T, rows, k, N, y_is_fp32 ? 1 : 0, out_is_fp32 ? 1 : 0};
    return cuda_status(sharq::launch_combine(p, static_cast<cudaStream_t>(stream)));
}

sharq_status sharq_residual_norm(const sharq_residual_norm_args* a, void* stream) {
    if (!a || !valid_norm_extent(a->M, a->K) || !valid_eps(a->eps) || !std::isfinite(a->alpha))
        return SHARQ_ERR_INVALID_ARG;
    if (a->norm < SHARQ_NORM_NONE || a->norm > SHARQ_NORM_LAYER) return SHARQ_ERR_INVALID_ARG;
    if (a->M > 0 && !a->x) return SHARQ_ERR_INVALID_ARG;
    if (a->M > 0 && !a->h && (a->post_gamma || a->gate)) return SHARQ_ERR_INVALID_ARG;
    if (a->norm == SHARQ_NORM_NONE && (a->gamma || a->beta || a->scale || a->shift)) return SHARQ_ERR_INVALID_ARG;
    if (a->G < 1 || (a->M > 0 && a->M % a->G != 0)) return SHARQ_ERR_INVALID_ARG;
    const int xs = a->x_is_fp32 ? 4 : 2, hs = a->h_is_fp32 ? 4 : 2, ms = a->mod_is_fp32 ? 4 : 2;
    if (!valid_ld(a->ld_x, a->K, a->M, xs) || (a->h && !valid_ld(a->ld_h, a->K, a->M, hs)) ||
        (a->out_x && !valid_ld(a->ld_out, a->K, a->M, xs)) || (a->gate && !valid_ld(a->ld_gate, a->K, a->G, ms)) ||
        (a->scale && !valid_ld(a->ld_scale, a->K, a->G, ms)) || (a->shift && !valid_ld(a->ld_shift, a->K, a->G, ms)))
        return SHARQ_ERR_INVALID_ARG;
    const void* all[] = {a->x, a->h, a->post_gamma, a->gate, a->gamma, a->beta, a->scale, a->shift, a->out_x, a->y};
    for (const void* p : all)
        if (!aligned(p, 16)) return SHARQ_ERR_INVALID_ARG;
    if (a->q && (a->q->M != a->M || a->q->K != a->K || !valid_rows8(a->q->codes, a->q->scales, a->M)))
        return SHARQ_ERR_INVALID_ARG;
    if (a->M == 0) return SHARQ_OK;
    sharq::NormLaunch p{};
    p.x = a->x; p.h = a->h; p.post_gamma = a->post_gamma; p.gate = a->gate; p.gamma = a->gamma; p.beta = a->beta;
    p.scale = a->scale; p.shift = a->shift; p.out_x = a->out_x; p.y = a->y;
    p.codes = a->q ? a->q->codes : nullptr; p.row_scale = a->q ? a->q->scales : nullptr;
    p.ldx = a->ld_x; p.ldh = a->ld_h; p.ld_gate = a->ld_gate; p.ld_scale = a->ld_scale; p.ld_shift = a->ld_shift;
    p.ldo = a->ld_out; p.M = a->M; p.group_rows = a->M / a->G; p.K = a->K; p.norm = a->norm;
    p.x_fp32 = a->x_is_fp32 ? 1 : 0; p.h_fp32 = a->h_is_fp32 ? 1 : 0; p.norm_fp32 = a->norm_is_fp32 ? 1 : 0;
    p.mod_fp32 = a->mod_is_fp32 ? 1 : 0; p.alpha = a->alpha; p.eps = a->eps;
    return cuda_status(sharq::launch_residual_norm(p, static_cast<cudaStream_t>(stream), sharq::device_sm_count()));
}

sharq_status sharq_prepare_int8(const void* X_bf16, const void* gamma_bf16, float eps,
                                const sharq_prepared_int8* out, void* stream) {
    if (!out) return SHARQ_ERR_INVALID_ARG;
    return quantize_rows(X_bf16, gamma_bf16, eps, out->codes, out->scales, out->M, out->K, stream);
}

sharq_status sharq_quantize_weight_int8(const void* W_bf16, const sharq_weight_int8* out, void* stream) {
    if (!out || out->N < 1) return SHARQ_ERR_INVALID_ARG;
    return quantize_rows(W_bf16, nullptr, 0.0f, out->codes, out->scales, out->N, out->K, stream);
}

sharq_status sharq_linear_int8(const sharq_prepared_int8* x, const sharq_weight_int8* w, const void* bias,
                               int bias_is_fp32, void* Y, int y_is_fp32, void* stream) {
    if (!x || !w || x->M < 0 || x->M > kMaxRows8 || w->N < 1 || w->N > kMaxRows8 || x->K != w->K || w->K < 16 || w->K > 65536 ||
        w->K % 16 != 0)
        return SHARQ_ERR_INVALID_ARG;
    if (!valid_rows8(x->codes, x->scales, x->M) || !valid_rows8(w->codes, w->scales, w->N))
        return SHARQ_ERR_INVALID_ARG;
    if ((x->M > 0 && !Y) || !aligned(Y, 16) || !aligned(bias, bias_is_fp32 ? 4 : 2)) return SHARQ_ERR_INVALID_ARG;
    if (x->M == 0) return SHARQ_OK;
    sharq::Int8Launch p{x->codes, x->scales, w->codes, w->scales, bias, Y, x->M, w->N, w->K,
                        bias_is_fp32 ? 1 : 0, y_is_fp32 ? 1 : 0};
    return cuda_status(sharq::launch_linear_int8(p, static_cast<cudaStream_t>(stream), sharq::device_sm_count()));
}

}  // extern "C"
