// losses.h -- the training objectives over rows of logits: what the entry
// points (api_losses.cu) hand to the kernels (losses.cu).
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

namespace lik {

enum LossHead : int { kHeadDistill = 0, kHeadPolicy = 1, kHeadToken = 2 };
// What a launch does with a row: statistics and loss; the gradient from saved
// statistics; both.
enum LossForm : int { kFwd = 0, kBwd = 1, kStep = 2 };

constexpr int kMaxTeacher = 1024;  // teacher entries per row

// One call over logits [rows, cols].  A target head (policy, token) has
// target and not the teacher's fields, and the other way round.
struct LossRows {
    const void* logits = nullptr;
    void* grad = nullptr;  // nullptr: no gradient
    int dtype = 0;
    int64_t rows = 0, cols = 0, stride = 0, grad_stride = 0;
    float scale = 1.0f;
    float c = 0.0f;  // scale * log2(e), rounded
    const float* weight = nullptr;  // [rows] or nullptr: even_weight each
    float even_weight = 0.0f;
    // distillation
    const int32_t* t_index = nullptr;  // [rows, k]
    const void* t_logits = nullptr;    // [rows, k] of t_dtype
    int t_dtype = 0;
    int k = 0;
    const float* t_lse = nullptr;  // [rows] or nullptr: normalised over the entries
    // target heads
    const int32_t* target = nullptr;  // [rows]
    const float* old_logp = nullptr;
    const float* advantage = nullptr;
    const float* ref_logp = nullptr;  // nullptr: no KL term
    float clip_low = 0.0f, clip_high = 0.0f, kl_coef = 0.0f;
    // outputs
    float* row_loss = nullptr;
    float* row_logp = nullptr;
    // (max, 1 / sum, log-probability or weight, coefficient or teacher mass);
    // 1 / sum is 0 for a row left out
    float4* state = nullptr;
    const float* grad_loss = nullptr;  // upstream gradient, backward only; nullptr: 1
    // Gradient of a target head: also *sum_out = the weighted sum of sum_value (as launch_loss_sum).
    // Forward and step of the distillation and policy heads: *sum_out may be written as the weighted
    // sum of row_loss, where launch_loss_rows says so.
    const float* sum_value = nullptr;
    const float* sum_weight = nullptr;
    int64_t sum_n = 0;
    float* sum_out = nullptr;
};

// The pairs of a preference loss, over the row states of a token-head forward.
struct LossPairs {
    int64_t rows = 0, pairs = 0;
    const int32_t* offsets = nullptr;  // [2 * pairs + 1]
    const float* ref_logp = nullptr;   // [2 * pairs] or nullptr
    const float* weight = nullptr;     // [pairs] or nullptr: 1 / pairs each
    float beta = 0.0f, margin = 0.0f, smoothing = 0.0f;
    bool average = false;
    float* pair_loss = nullptr;
    float* seq_logp = nullptr;
    float4* state = nullptr;  // [rows]: reads 1 / sum and the log-probability, writes the coefficient
};

// Forward (row losses or log-probabilities, and row states unless nullptr);
// with L.grad set, forward and gradient in one launch.  *summed (unless
// nullptr): whether it also wrote *L.sum_out.
cudaError_t launch_loss_rows(LossHead head, const LossRows& L, bool* summed, cudaStream_t stream);

// Gradient from the row states of a forward.
cudaError_t launch_loss_grad(LossHead head, const LossRows& L, cudaStream_t stream);

// Sequence sums, pair losses and every row's coefficient.
cudaError_t launch_loss_pairs(const LossPairs& P, cudaStream_t stream);

// *loss = sum of weight * value over n values, in a fixed order (weight
// nullptr: 1 / n each); a value of 0 adds nothing whatever its weight.
cudaError_t launch_loss_sum(const float* value, const float* weight, int64_t n, float* loss, cudaStream_t stream);

}  // namespace lik
