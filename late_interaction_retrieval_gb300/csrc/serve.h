// serve.h -- a serving step over a cache in 8 bits: what the entry points
// (api_serve.cu) hand to the kernels (cache_slots.cu, cache_write.cu,
// cache_attention.cu, verify.cu).
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

namespace lik {

constexpr int kMaxRequests = 8192;
constexpr int kMaxHeadDim = 128;
constexpr float kCodeMax = 448.0f;             // largest e4m3 value
constexpr float kLeastScale = 1.17549435e-38f;  // 2^-126

struct SlotsArgs {
    const int32_t *cached, *added, *held;
    int requests;
    int page_shift;
    const int32_t* free_pages;
    int64_t free_capacity;
    const int32_t* free_count;
    int32_t* table;
    int64_t cols, stride;
    int32_t *held_out, *lengths, *offsets;
    int64_t* slots;
    int64_t capacity;
    int32_t* free_left;
    int32_t *most, *missing;  // whether the step fits: both, or neither
};
cudaError_t launch_cache_slots(const SlotsArgs& a, cudaStream_t stream);

struct WriteArgs {
    const void* x[2];  // keys, values
    int dtype;
    int64_t rows;
    int heads, dim;
    int64_t token_stride[2], head_stride[2];
    const int64_t* slots;
    uint8_t* cache[2];
    float* scale[2];
    int64_t pages;
    int page_shift;
};
cudaError_t launch_cache_write(const WriteArgs& a, cudaStream_t stream);

struct AttentionArgs {
    const void* q;
    int dtype;
    int64_t rows;
    int q_heads, heads, dim;
    int64_t q_token_stride, q_head_stride;
    const uint8_t *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    int64_t pages;
    int page_shift;
    const int32_t* table;
    int64_t cols, stride;
    const int32_t *offsets, *lengths;
    int requests;
    int64_t max_added;
    float scale;
    void* out;
    int64_t out_token_stride, out_head_stride;
    float* lse;
    void* workspace;
};
size_t cache_attention_workspace(int64_t rows, int64_t q_heads, int64_t heads, int64_t dim, int64_t requests,
                                 int64_t max_added);
cudaError_t launch_cache_attention(const AttentionArgs& a, cudaStream_t stream);

struct VerifyArgs {
    const void *target, *draft;  // draft nullptr: one-hot drafts
    int dtype;
    int64_t drafts;
    int requests;
    int64_t cols, target_stride, draft_stride;
    const int32_t *drafted, *offsets;
    const float *uniform, *noise;
    float scale;
    int32_t *tokens, *accepted;
    float* logp;
    void* workspace;
};
size_t verify_workspace(int64_t drafts, int64_t requests, int64_t cols);
cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t stream);

}  // namespace lik
