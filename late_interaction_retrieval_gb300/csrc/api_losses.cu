// api_losses.cu -- C entry points of the training objectives over logits
// (include/lik.h): argument checks and the launches of each form.
#include <cmath>

#include "lik.h"
#include "lik_internal.h"
#include "losses.h"
#include "validate.h"

namespace lik {
namespace {

size_t elem_bytes(lik_dtype t) { return t == LIK_F32 ? 4 : 2; }

// Elements from the first row's start to the last row's end.
int64_t span(int64_t rows, int64_t cols, int64_t stride) { return rows > 0 ? (rows - 1) * stride + cols : 0; }

// Keeps every byte offset far inside 64 bits; no buffer is as large.
constexpr int64_t kMaxSpan = int64_t(1) << 48;

lik_status check_rows(lik_dtype dtype, int64_t rows, int64_t cols, int64_t row_stride, float scale) {
    if (!known_dtype(dtype)) return fail(LIK_ERR_INVALID_ARG, "unknown dtype %d", static_cast<int>(dtype));
    if (rows < 0 || cols < 0) return fail(LIK_ERR_INVALID_ARG, "negative size");
    if (cols < 1) return fail(LIK_ERR_INVALID_ARG, "cols must be >= 1");
    if (rows > INT32_MAX) return fail(LIK_ERR_UNSUPPORTED, "rows %lld > 2^31 - 1", static_cast<long long>(rows));
    if (cols > (int64_t(1) << 30)) return fail(LIK_ERR_UNSUPPORTED, "cols %lld > 2^30", static_cast<long long>(cols));
    if (row_stride < cols)
        return fail(LIK_ERR_INVALID_ARG, "row_stride %lld < cols %lld", static_cast<long long>(row_stride),
                    static_cast<long long>(cols));
    if (row_stride > (int64_t(1) << 31))
        return fail(LIK_ERR_UNSUPPORTED, "row_stride %lld > 2^31", static_cast<long long>(row_stride));
    if (span(rows, cols, row_stride) > kMaxSpan) return fail(LIK_ERR_UNSUPPORTED, "logits span more than 2^48 elements");
    if (!(scale >= 1e-30f && scale <= 1e30f))
        return fail(LIK_ERR_INVALID_ARG, "scale must lie in [1e-30, 1e30] (got %g)", static_cast<double>(scale));
    return LIK_OK;
}

lik_status check_grad(lik_dtype dtype, int64_t rows, int64_t cols, const void* logits, int64_t row_stride,
                      const void* grad, int64_t grad_stride) {
    if (grad_stride < cols)
        return fail(LIK_ERR_INVALID_ARG, "grad_stride %lld < cols %lld", static_cast<long long>(grad_stride),
                    static_cast<long long>(cols));
    if (grad_stride > (int64_t(1) << 31))
        return fail(LIK_ERR_UNSUPPORTED, "grad_stride %lld > 2^31", static_cast<long long>(grad_stride));
    if (span(rows, cols, grad_stride) > kMaxSpan)
        return fail(LIK_ERR_UNSUPPORTED, "grad_logits spans more than 2^48 elements");
    if (rows == 0) return LIK_OK;
    const uintptr_t z0 = reinterpret_cast<uintptr_t>(logits), g0 = reinterpret_cast<uintptr_t>(grad);
    const uintptr_t z1 = z0 + span(rows, cols, row_stride) * elem_bytes(dtype);
    const uintptr_t g1 = g0 + span(rows, cols, grad_stride) * elem_bytes(dtype);
    if (z0 < g1 && g0 < z1 && !(z0 == g0 && (row_stride == grad_stride || rows == 1)))
        return fail(LIK_ERR_INVALID_ARG,
                    "grad_logits overlaps logits: it must be the logits buffer itself (same address and stride) or "
                    "lie apart from it");
    return LIK_OK;
}

lik_status check_aligns(lik_dtype dtype, const void* logits, const void* grad, const void* state) {
    lik_status st = check_aligned(logits, elem_bytes(dtype), "logits");
    if (st == LIK_OK) st = check_aligned(grad, elem_bytes(dtype), "grad_logits");
    if (st == LIK_OK) st = check_aligned(state, 16, "row_state");
    return st;
}

// Every other buffer holds 4-byte elements (teacher logits may hold 2-byte ones).
lik_status check_four(const Spec* specs, int n) {
    for (int i = 0; i < n; ++i) {
        const lik_status st = check_aligned(specs[i].ptr, 4, specs[i].name);
        if (st != LIK_OK) return st;
    }
    return LIK_OK;
}

LossRows make_rows(const void* logits, lik_dtype dtype, int64_t rows, int64_t cols, int64_t row_stride, float scale) {
    LossRows L;
    L.logits = logits;
    L.dtype = static_cast<int>(dtype);
    L.rows = rows;
    L.cols = cols;
    L.stride = row_stride;
    L.scale = scale;
    L.c = static_cast<float>(static_cast<double>(scale) * 1.4426950408889634074);
    L.even_weight = rows > 0 ? 1.0f / static_cast<float>(rows) : 0.0f;
    return L;
}

struct DistillArgs {
    const void* logits;
    lik_dtype dtype;
    int64_t rows, cols, row_stride;
    const int32_t* index;
    const void* teacher;
    lik_dtype teacher_dtype;
    int64_t k;
    const float* lse;
    const float* weight;
    float scale;
};

lik_status distill(const DistillArgs& a, float* loss, float* row_loss, float* row_state, const float* grad_loss,
                   void* grad, int64_t grad_stride, bool fwd, bool bwd, cudaStream_t stream) {
    clear_message();
    lik_status st = check_rows(a.dtype, a.rows, a.cols, a.row_stride, a.scale);
    if (st != LIK_OK) return st;
    if (!known_dtype(a.teacher_dtype))
        return fail(LIK_ERR_INVALID_ARG, "unknown teacher_dtype %d", static_cast<int>(a.teacher_dtype));
    if (a.k < 0) return fail(LIK_ERR_INVALID_ARG, "negative size");
    if (a.k > kMaxTeacher)
        return fail(LIK_ERR_UNSUPPORTED, "k %lld > %d", static_cast<long long>(a.k), kMaxTeacher);
    if (bwd && (st = check_grad(a.dtype, a.rows, a.cols, a.logits, a.row_stride, grad, grad_stride)) != LIK_OK)
        return st;
    int dev = 0;
    if ((st = check_device(&dev)) != LIK_OK) return st;
    const Spec specs[] = {
        {"logits", a.logits, true, span(a.rows, a.cols, a.row_stride)},
        {"grad_logits", grad, bwd, bwd ? span(a.rows, a.cols, grad_stride) : 0},
        {"teacher_logits", a.teacher, true, a.rows * a.k},
        {"teacher_index", a.index, true, a.rows * a.k},
        {"teacher_lse", a.lse, false, a.rows},
        {"row_weight", a.weight, false, a.rows},
        {"loss", loss, fwd, fwd ? 1 : 0},
        {"row_loss", row_loss, fwd, fwd ? a.rows : 0},
        {"row_state", row_state, !fwd, a.rows},
        {"grad_loss", grad_loss, false, 1},
    };
    if ((st = check_buffers(dev, specs, 10)) != LIK_OK) return st;
    if ((st = check_four(specs + 3, 7)) != LIK_OK) return st;
    if ((st = check_aligned(a.teacher, elem_bytes(a.teacher_dtype), "teacher_logits")) != LIK_OK) return st;
    if ((st = check_aligns(a.dtype, a.logits, grad, row_state)) != LIK_OK) return st;
    LossRows L = make_rows(a.logits, a.dtype, a.rows, a.cols, a.row_stride, a.scale);
    L.weight = a.weight;
    L.t_index = a.index;
    L.t_logits = a.teacher;
    L.t_dtype = static_cast<int>(a.teacher_dtype);
    L.k = static_cast<int>(a.k);
    L.t_lse = a.lse;
    L.row_loss = row_loss;
    L.state = reinterpret_cast<float4*>(row_state);
    L.grad_loss = grad_loss;
    if (bwd) {
        L.grad = grad;
        L.grad_stride = grad_stride;
    }
    cudaError_t e = cudaSuccess;
    if (fwd) {
        bool summed = false;
        L.sum_out = loss;
        if (a.rows > 0) e = launch_loss_rows(kHeadDistill, L, &summed, stream);
        if (e == cudaSuccess && !summed) e = launch_loss_sum(row_loss, a.weight, a.rows, loss, stream);
    } else if (a.rows > 0) {
        e = launch_loss_grad(kHeadDistill, L, stream);
    }
    return e == cudaSuccess ? LIK_OK : cuda_fail(e, "distillation launch");
}

struct PolicyArgs {
    const void* logits;
    lik_dtype dtype;
    int64_t rows, cols, row_stride;
    const int32_t* target;
    const float *old_logp, *advantage, *ref_logp, *weight;
    float clip_low, clip_high, kl_coef, scale;
};

lik_status policy(const PolicyArgs& a, float* loss, float* row_loss, float* row_logp, float* row_state, void* grad,
                  int64_t grad_stride, bool bwd, cudaStream_t stream) {
    clear_message();
    lik_status st = check_rows(a.dtype, a.rows, a.cols, a.row_stride, a.scale);
    if (st != LIK_OK) return st;
    if (!(a.clip_low >= 0.0f && a.clip_low <= 1.0f) || !(a.clip_high >= 0.0f) || !std::isfinite(a.clip_high))
        return fail(LIK_ERR_INVALID_ARG, "clip_low must lie in [0, 1] and clip_high be >= 0 and finite (got %g, %g)",
                    static_cast<double>(a.clip_low), static_cast<double>(a.clip_high));
    if (!std::isfinite(a.kl_coef)) return fail(LIK_ERR_INVALID_ARG, "kl_coef must be finite");
    if (bwd && (st = check_grad(a.dtype, a.rows, a.cols, a.logits, a.row_stride, grad, grad_stride)) != LIK_OK)
        return st;
    int dev = 0;
    if ((st = check_device(&dev)) != LIK_OK) return st;
    const Spec specs[] = {
        {"logits", a.logits, true, span(a.rows, a.cols, a.row_stride)},
        {"grad_logits", grad, bwd, bwd ? span(a.rows, a.cols, grad_stride) : 0},
        {"target", a.target, true, a.rows},
        {"old_logp", a.old_logp, true, a.rows},
        {"advantage", a.advantage, true, a.rows},
        {"ref_logp", a.ref_logp, false, a.rows},
        {"row_weight", a.weight, false, a.rows},
        {"loss", loss, true, 1},
        {"row_loss", row_loss, true, a.rows},
        {"row_logp", row_logp, true, a.rows},
        {"row_state", row_state, false, a.rows},
    };
    if ((st = check_buffers(dev, specs, 11)) != LIK_OK) return st;
    if ((st = check_four(specs + 2, 9)) != LIK_OK) return st;
    if ((st = check_aligns(a.dtype, a.logits, grad, row_state)) != LIK_OK) return st;
    LossRows L = make_rows(a.logits, a.dtype, a.rows, a.cols, a.row_stride, a.scale);
    L.weight = a.weight;
    L.target = a.target;
    L.old_logp = a.old_logp;
    L.advantage = a.advantage;
    L.ref_logp = a.kl_coef != 0.0f ? a.ref_logp : nullptr;  // no term, and no 0 * inf of a far reference
    L.clip_low = a.clip_low;
    L.clip_high = a.clip_high;
    L.kl_coef = a.kl_coef;
    L.row_loss = row_loss;
    L.row_logp = row_logp;
    L.state = reinterpret_cast<float4*>(row_state);
    if (bwd) {
        L.grad = grad;
        L.grad_stride = grad_stride;
    }
    cudaError_t e = cudaSuccess;
    bool summed = false;
    L.sum_out = loss;
    if (a.rows > 0) e = launch_loss_rows(kHeadPolicy, L, &summed, stream);
    if (e == cudaSuccess && !summed) e = launch_loss_sum(row_loss, a.weight, a.rows, loss, stream);
    return e == cudaSuccess ? LIK_OK : cuda_fail(e, "policy loss launch");
}

// The gradient of a target head from its row states (policy and preference).
lik_status target_bwd(LossHead head, const void* logits, lik_dtype dtype, int64_t rows, int64_t cols,
                      int64_t row_stride, const int32_t* target, float scale, const float* row_state,
                      const float* grad_loss, void* grad, int64_t grad_stride, cudaStream_t stream) {
    clear_message();
    lik_status st = check_rows(dtype, rows, cols, row_stride, scale);
    if (st != LIK_OK) return st;
    if ((st = check_grad(dtype, rows, cols, logits, row_stride, grad, grad_stride)) != LIK_OK) return st;
    int dev = 0;
    if ((st = check_device(&dev)) != LIK_OK) return st;
    const Spec specs[] = {
        {"logits", logits, true, span(rows, cols, row_stride)},
        {"grad_logits", grad, true, span(rows, cols, grad_stride)},
        {"target", target, true, rows},
        {"row_state", row_state, true, rows},
        {"grad_loss", grad_loss, false, 1},
    };
    if ((st = check_buffers(dev, specs, 5)) != LIK_OK) return st;
    if ((st = check_four(specs + 2, 3)) != LIK_OK) return st;
    if ((st = check_aligns(dtype, logits, grad, row_state)) != LIK_OK) return st;
    if (rows == 0) return LIK_OK;
    LossRows L = make_rows(logits, dtype, rows, cols, row_stride, scale);
    L.target = target;
    L.state = reinterpret_cast<float4*>(const_cast<float*>(row_state));
    L.grad_loss = grad_loss;
    L.grad = grad;
    L.grad_stride = grad_stride;
    const cudaError_t e = launch_loss_grad(head, L, stream);
    return e == cudaSuccess ? LIK_OK : cuda_fail(e, "gradient launch");
}

struct PreferenceArgs {
    const void* logits;
    lik_dtype dtype;
    int64_t rows, cols, row_stride;
    const int32_t *target, *offsets;
    int64_t pairs;
    const float *ref_logp, *weight;
    float beta, margin, smoothing;
    int average;
    float scale;
};

lik_status preference(const PreferenceArgs& a, float* loss, float* pair_loss, float* seq_logp, float* row_state,
                      void* grad, int64_t grad_stride, bool bwd, cudaStream_t stream) {
    clear_message();
    lik_status st = check_rows(a.dtype, a.rows, a.cols, a.row_stride, a.scale);
    if (st != LIK_OK) return st;
    if (a.pairs < 0) return fail(LIK_ERR_INVALID_ARG, "negative size");
    if (a.pairs > (int64_t(1) << 20))
        return fail(LIK_ERR_UNSUPPORTED, "pairs %lld > 2^20", static_cast<long long>(a.pairs));
    if (!std::isfinite(a.beta) || !std::isfinite(a.margin))
        return fail(LIK_ERR_INVALID_ARG, "beta and margin must be finite");
    if (!(a.smoothing >= 0.0f && a.smoothing <= 1.0f))
        return fail(LIK_ERR_INVALID_ARG, "smoothing must lie in [0, 1] (got %g)", static_cast<double>(a.smoothing));
    if (bwd && (st = check_grad(a.dtype, a.rows, a.cols, a.logits, a.row_stride, grad, grad_stride)) != LIK_OK)
        return st;
    int dev = 0;
    if ((st = check_device(&dev)) != LIK_OK) return st;
    const Spec specs[] = {
        {"logits", a.logits, true, span(a.rows, a.cols, a.row_stride)},
        {"grad_logits", grad, bwd, bwd ? span(a.rows, a.cols, grad_stride) : 0},
        {"target", a.target, true, a.rows},
        {"offsets", a.offsets, true, 2 * a.pairs + 1},
        {"ref_logp", a.ref_logp, false, 2 * a.pairs},
        {"pair_weight", a.weight, false, a.pairs},
        {"loss", loss, true, 1},
        {"pair_loss", pair_loss, true, a.pairs},
        {"seq_logp", seq_logp, true, 2 * a.pairs},
        {"row_state", row_state, true, a.rows},
    };
    if ((st = check_buffers(dev, specs, 10)) != LIK_OK) return st;
    if ((st = check_four(specs + 2, 8)) != LIK_OK) return st;
    if ((st = check_aligns(a.dtype, a.logits, grad, row_state)) != LIK_OK) return st;
    LossRows L = make_rows(a.logits, a.dtype, a.rows, a.cols, a.row_stride, a.scale);
    L.target = a.target;
    L.state = reinterpret_cast<float4*>(row_state);
    LossPairs P;
    P.rows = a.rows;
    P.pairs = a.pairs;
    P.offsets = a.offsets;
    P.ref_logp = a.ref_logp;
    P.weight = a.weight;
    P.beta = a.beta;
    P.margin = a.margin;
    P.smoothing = a.smoothing;
    P.average = a.average != 0;
    P.pair_loss = pair_loss;
    P.seq_logp = seq_logp;
    P.state = L.state;
    cudaError_t e = cudaSuccess;
    const bool grad_rows = bwd && a.rows > 0;
    if (a.rows > 0) e = launch_loss_rows(kHeadToken, L, nullptr, stream);
    if (e == cudaSuccess && a.pairs > 0) e = launch_loss_pairs(P, stream);
    if (e == cudaSuccess && grad_rows) {  // sums the loss on the way
        L.grad = grad;
        L.grad_stride = grad_stride;
        L.sum_value = pair_loss;
        L.sum_weight = a.weight;
        L.sum_n = a.pairs;
        L.sum_out = loss;
        e = launch_loss_grad(kHeadToken, L, stream);
    } else if (e == cudaSuccess) {
        e = launch_loss_sum(pair_loss, a.weight, a.pairs, loss, stream);
    }
    return e == cudaSuccess ? LIK_OK : cuda_fail(e, "preference loss launch");
}

}  // namespace
}  // namespace lik

using namespace lik;

extern "C" {

lik_status lik_distill_topk_fwd(const void* logits, lik_dtype dtype, int64_t rows, int64_t cols, int64_t row_stride,
                                const int32_t* teacher_index, const void* teacher_logits, lik_dtype teacher_dtype,
                                int64_t k, const float* teacher_lse, const float* row_weight, float scale,
                                float* loss, float* row_loss, float* row_state, cudaStream_t stream) {
    return distill({logits, dtype, rows, cols, row_stride, teacher_index, teacher_logits, teacher_dtype, k,
                    teacher_lse, row_weight, scale},
                   loss, row_loss, row_state, nullptr, nullptr, 0, true, false, stream);
}

lik_status lik_distill_topk_bwd(const void* logits, lik_dtype dtype, int64_t rows, int64_t cols, int64_t row_stride,
                                const int32_t* teacher_index, const void* teacher_logits, lik_dtype teacher_dtype,
                                int64_t k, const float* teacher_lse, float scale, const float* row_state,
                                const float* grad_loss, void* grad_logits, int64_t grad_stride,
                                cudaStream_t stream) {
    return distill({logits, dtype, rows, cols, row_stride, teacher_index, teacher_logits, teacher_dtype, k,
                    teacher_lse, nullptr, scale},
                   nullptr, nullptr, const_cast<float*>(row_state), grad_loss, grad_logits, grad_stride, false, true,
                   stream);
}

lik_status lik_distill_topk_step(const void* logits, lik_dtype dtype, int64_t rows, int64_t cols,
                                 int64_t row_stride, const int32_t* teacher_index, const void* teacher_logits,
                                 lik_dtype teacher_dtype, int64_t k, const float* teacher_lse,
                                 const float* row_weight, float scale, float* loss, float* row_loss,
                                 void* grad_logits, int64_t grad_stride, cudaStream_t stream) {
    return distill({logits, dtype, rows, cols, row_stride, teacher_index, teacher_logits, teacher_dtype, k,
                    teacher_lse, row_weight, scale},
                   loss, row_loss, nullptr, nullptr, grad_logits, grad_stride, true, true, stream);
}

lik_status lik_policy_loss_fwd(const void* logits, lik_dtype dtype, int64_t rows, int64_t cols, int64_t row_stride,
                               const int32_t* target, const float* old_logp, const float* advantage,
                               const float* ref_logp, const float* row_weight, float clip_low, float clip_high,
                               float kl_coef, float scale, float* loss, float* row_loss, float* row_logp,
                               float* row_state, cudaStream_t stream) {
    return policy({logits, dtype, rows, cols, row_stride, target, old_logp, advantage, ref_logp, row_weight, clip_low,
                   clip_high, kl_coef, scale},
                  loss, row_loss, row_logp, row_state, nullptr, 0, false, stream);
}

lik_status lik_policy_loss_bwd(const void* logits, lik_dtype dtype, int64_t rows, int64_t cols, int64_t row_stride,
                               const int32_t* target, float scale, const float* row_state, const float* grad_loss,
                               void* grad_logits, int64_t grad_stride, cudaStream_t stream) {
    return target_bwd(kHeadPolicy, logits, dtype, rows, cols, row_stride, target, scale, row_state, grad_loss,
                      grad_logits, grad_stride, stream);
}

lik_status lik_policy_loss_step(const void* logits, lik_dtype dtype, int64_t rows, int64_t cols, int64_t row_stride,
                                const int32_t* target, const float* old_logp, const float* advantage,
                                const float* ref_logp, const float* row_weight, float clip_low, float clip_high,
                                float kl_coef, float scale, float* loss, float* row_loss, float* row_logp,
                                void* grad_logits, int64_t grad_stride, cudaStream_t stream) {
    return policy({logits, dtype, rows, cols, row_stride, target, old_logp, advantage, ref_logp, row_weight, clip_low,
                   clip_high, kl_coef, scale},
                  loss, row_loss, row_logp, nullptr, grad_logits, grad_stride, true, stream);
}

lik_status lik_preference_loss_fwd(const void* logits, lik_dtype dtype, int64_t rows, int64_t cols,
                                   int64_t row_stride, const int32_t* target, const int32_t* offsets, int64_t pairs,
                                   const float* ref_logp, const float* pair_weight, float beta, float margin,
                                   float smoothing, int average, float scale, float* loss, float* pair_loss,
                                   float* seq_logp, float* row_state, cudaStream_t stream) {
    return preference({logits, dtype, rows, cols, row_stride, target, offsets, pairs, ref_logp, pair_weight, beta,
                       margin, smoothing, average, scale},
                      loss, pair_loss, seq_logp, row_state, nullptr, 0, false, stream);
}

lik_status lik_preference_loss_bwd(const void* logits, lik_dtype dtype, int64_t rows, int64_t cols,
                                   int64_t row_stride, const int32_t* target, float scale, const float* row_state,
                                   const float* grad_loss, void* grad_logits, int64_t grad_stride,
                                   cudaStream_t stream) {
    return target_bwd(kHeadToken, logits, dtype, rows, cols, row_stride, target, scale, row_state, grad_loss,
                      grad_logits, grad_stride, stream);
}

lik_status lik_preference_loss_step(const void* logits, lik_dtype dtype, int64_t rows, int64_t cols,
                                    int64_t row_stride, const int32_t* target, const int32_t* offsets, int64_t pairs,
                                    const float* ref_logp, const float* pair_weight, float beta, float margin,
                                    float smoothing, int average, float scale, float* loss, float* pair_loss,
                                    float* seq_logp, float* row_state, void* grad_logits, int64_t grad_stride,
                                    cudaStream_t stream) {
    return preference({logits, dtype, rows, cols, row_stride, target, offsets, pairs, ref_logp, pair_weight, beta,
                       margin, smoothing, average, scale},
                      loss, pair_loss, seq_logp, row_state, grad_logits, grad_stride, true, stream);
}

}  // extern "C"
