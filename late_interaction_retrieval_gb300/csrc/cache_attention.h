// cache_attention.h -- what the kernels of attention over the 8-bit cache share.
#pragma once

#include <atomic>

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "lik_internal.h"
#include "serve.h"
#include "sm100_ptx.cuh"

namespace lik {
namespace attn {

// log2 of the largest weight, and of a row's largest one when its reference is set; the reference that a row
// which has seen nothing has where sums are joined (below any other; its own sum is 0).
constexpr float kLogTop = 15.0f, kLogStart = 7.0f, kNothing = -1.70141183e38f;

// One request as the device has it, clamped to what the buffers hold.
struct Request {
    int row0, n;   // its rows
    int length;    // its tokens in the cache, as far as its table goes
    int before;    // its tokens before the first row's, wherever they are: row i sees before + i + 1
};

__device__ __forceinline__ Request request_of(const AttentionArgs& a, int b) {
    Request r;
    const int rows = static_cast<int>(a.rows);
    int lo = a.offsets[b], hi = a.offsets[b + 1];
    lo = min(max(lo, 0), rows);
    hi = min(max(hi, lo), rows);
    r.row0 = lo;
    r.n = hi - lo;
    // A request that is longer than its table: the tokens behind it are hidden, and the rows stay where they are.
    const int all = max(a.lengths[b], 0);
    r.length = min(all, static_cast<int>(a.cols << a.page_shift));
    r.before = all - r.n;
    return r;
}

// Two e4m3 codes (low byte first) of a word's lower or upper half as fp16:
// exact, NaN stays NaN.
__device__ __forceinline__ uint32_t widen_low(uint32_t codes) {
    uint32_t h;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}" : "=r"(h) : "r"(codes));
    return h;
}
__device__ __forceinline__ uint32_t widen_high(uint32_t codes) {
    uint32_t h;
    asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}" : "=r"(h) : "r"(codes));
    return h;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The power of two that brings a row whose largest size is `most` to [2^14, 2^15).
__device__ __forceinline__ int row_shift(float most) {
    if (!(most > 0.0f) || most > 3.402823466e38f) return 0;
    return 14 - ilogbf(most);
}

// 2^shift in two factors, each a normal number for any shift that row_shift gives (or its negative).
__device__ __forceinline__ float2 power_of_two(int shift) {
    const int half = shift >> 1;
    return make_float2(__int_as_float((127 + half) << 23), __int_as_float((127 + shift - half) << 23));
}

__device__ __forceinline__ float2 widen_q(uint32_t v, bool bf16) {
    if (bf16) return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

__device__ __forceinline__ uint32_t pack_half(float x, float y) {
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// What the rounding to the two halves of h left of x and y.  An fp16 output holds 11 bits itself, so its weights' 11
// bits would show in it (half as much again as its own rounding): there a second product adds what is left.  A bf16
// output's 8 bits hide it.
__device__ __forceinline__ uint32_t left_of(uint32_t h, float x, float y) {
    const float2 got = __half22float2(*reinterpret_cast<const __half2*>(&h));
    return pack_half(x - got.x, y - got.y);
}

// Sets a kernel's shared-memory limit once for each device (`done`: one bit a device, of the kernel's own).
template <typename Kernel>
inline cudaError_t allow_shared(Kernel kernel, size_t bytes, int device, std::atomic<uint64_t>& done) {
    const uint64_t bit = uint64_t(1) << (device & 63);
    if (device < 64 && (done.load(std::memory_order_acquire) & bit)) return cudaSuccess;
    const cudaError_t e =
        cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
    if (e == cudaSuccess && device < 64) done.fetch_or(bit, std::memory_order_release);
    return e;
}

}  // namespace attn

cudaError_t launch_attention_split(const AttentionArgs& a, cudaStream_t stream);
size_t attention_split_workspace(int64_t dim, int sms);
cudaError_t launch_attention_wide(const AttentionArgs& a, cudaStream_t stream);
size_t attention_wide_workspace(int64_t rows, int64_t group, int64_t dim, int sms);

}  // namespace lik
