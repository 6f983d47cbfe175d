// cache_attention.cu -- attention of a batch's new tokens over the 8-bit cache.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "dtype_load.cuh"
#include "lik_internal.h"
#include "serve.h"

namespace lik {
namespace {

constexpr int kThreads = 128;

__device__ __forceinline__ float decode(uint32_t code) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3)));
}

__device__ __forceinline__ void store(__half* p, float x) { *p = __float2half_rn(x); }
__device__ __forceinline__ void store(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// One warp a row (token, query head); lane l holds the dimensions l, l + 32, ...
template <typename T>
__global__ void __launch_bounds__(kThreads) cache_attention_rows(const AttentionArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t item = blockIdx.x * static_cast<int64_t>(kThreads / 32) + (threadIdx.x >> 5);
    if (item >= a.rows * a.q_heads) return;
    const int64_t t = item / a.q_heads;
    const int h = static_cast<int>(item - t * a.q_heads), kv = h / (a.q_heads / a.heads);
    int lo = 0, hi = a.requests;  // the request with offsets[b] <= t < offsets[b + 1]
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (a.offsets[mid + 1] <= t) lo = mid + 1;
        else hi = mid;
    }
    if (lo == a.requests || a.offsets[lo] > t) return;
    const int page_size = 1 << a.page_shift;
    const int64_t n = a.offsets[lo + 1] - a.offsets[lo], i = t - a.offsets[lo];
    int64_t sees = a.lengths[lo] - n + i + 1;
    const int64_t room = a.cols << a.page_shift;
    sees = sees < room ? sees : room;
    const T* const q = static_cast<const T*>(a.q) + t * a.q_token_stride + h * a.q_head_stride;
    float qv[4], acc[4] = {0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < 4; ++k) qv[k] = lane + 32 * k < a.dim ? to_f32(q[lane + 32 * k]) : 0.0f;
    float m = -INFINITY, sum = 0.0f;
    for (int64_t j = 0; j < sees; ++j) {
        const int64_t page = a.table[lo * a.stride + (j >> a.page_shift)];
        if (page < 0 || page >= a.pages) continue;
        const int64_t at = (((page * a.heads + kv) << a.page_shift) + (j & (page_size - 1))) * a.dim;
        float s = 0.0f;
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (lane + 32 * k < a.dim) s += qv[k] * decode(a.k_cache[at + lane + 32 * k]);
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= a.scale * a.k_scale[page * a.heads + kv];
        const float top = fmaxf(m, s);
        const float keep = top == -INFINITY ? 0.0f : __expf(m - top), e = top == -INFINITY ? 0.0f : __expf(s - top);
        sum = sum * keep + e;
        const float w = e * a.v_scale[page * a.heads + kv];
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (lane + 32 * k < a.dim) acc[k] = acc[k] * keep + w * decode(a.v_cache[at + lane + 32 * k]);
        m = top;
    }
    T* const out = static_cast<T*>(a.out) + t * a.out_token_stride + h * a.out_head_stride;
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (lane + 32 * k < a.dim) store(out + lane + 32 * k, sum == 0.0f ? 0.0f : acc[k] / sum);
    if (lane == 0 && a.lse) a.lse[item] = sum == 0.0f ? -INFINITY : m + logf(sum);
}

template <typename T>
cudaError_t launch(const AttentionArgs& a, cudaStream_t stream) {
    const int64_t items = a.rows * a.q_heads, per = kThreads / 32;
    cache_attention_rows<T><<<static_cast<unsigned>((items + per - 1) / per), kThreads, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

size_t cache_attention_workspace(int64_t, int64_t, int64_t, int64_t, int64_t, int64_t) { return 16; }

cudaError_t launch_cache_attention(const AttentionArgs& a, cudaStream_t stream) {
    return a.dtype == kF16 ? launch<__half>(a, stream) : launch<__nv_bfloat16>(a, stream);
}

}  // namespace lik
