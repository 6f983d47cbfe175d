// cache_write.cu -- new keys and values into the 8-bit cache, one scale for
// each page and head.
//
// A run (rows of consecutive slots in one page) of one head is one block's
// work: its largest value gives the page's scale, and only then can it be
// rounded.  The block keeps the run in registers between the two, so that it
// is read once.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "dtype_load.cuh"
#include "lik_internal.h"
#include "serve.h"

namespace lik {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kKept = 8;  // vectors of 8 values that a thread keeps

template <typename T>
__device__ __forceinline__ void load8(const T* p, bool wide, T (&v)[8]) {
    if (wide) {
        constexpr int n = sizeof(T) * 8 / 16;
        const uint4* s = reinterpret_cast<const uint4*>(p);
        uint4* d = reinterpret_cast<uint4*>(v);
#pragma unroll
        for (int i = 0; i < n; ++i) d[i] = __ldg(s + i);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = p[i];
    }
}

__device__ __forceinline__ float finite_size(float x) {
    const float s = fabsf(x);
    return s <= 3.402823466e38f ? s : 0.0f;  // NaN and infinity do not count
}

// Two codes; what is not finite becomes NaN (the conversion alone would turn
// an infinity into the largest value).
__device__ __forceinline__ uint32_t code2(float x, float y) {
    x = fabsf(x) <= 3.402823466e38f ? x : __int_as_float(0x7fffffff);
    y = fabsf(y) <= 3.402823466e38f ? y : __int_as_float(0x7fffffff);
    return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float decode(uint32_t code) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3)));
}

// 8 values in units of their scale, as codes.  x * inverse may overflow only
// where x is not finite already: |x| <= 448 * scale up to rounding.
template <typename T>
__device__ __forceinline__ uint2 encode8(const T (&v)[8], float inverse) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = code2(to_f32(v[2 * i]) * inverse, to_f32(v[2 * i + 1]) * inverse);
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

template <typename T>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const WriteArgs a, int chunk, bool wide_k, bool wide_v) {
    __shared__ float warp_max[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int head = blockIdx.y, which = blockIdx.z;
    const bool wide = which ? wide_v : wide_k;
    const T* const x = static_cast<const T*>(a.x[which]) + head * a.head_stride[which];
    const int64_t token_stride = a.token_stride[which];
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * chunk;
    const int64_t t1 = t0 + chunk < a.rows ? t0 + chunk : a.rows;
    const int page_size = 1 << a.page_shift;
    const int64_t n_slots = a.pages << a.page_shift;
    const int per_row = a.dim / 8;
    const float inv_row = 1.0f / static_cast<float>(per_row);

    for (int64_t t = t0; t < t1;) {
        const int64_t slot = a.slots[t];
        const int64_t before = t > 0 ? a.slots[t - 1] : -2;
        const int offset = static_cast<int>(slot & (page_size - 1));
        if (slot < 0 || slot >= n_slots || (before + 1 == slot && before >= 0 && offset != 0)) {
            ++t;  // no slot, or inside the run of a row before it
            continue;
        }
        // the run's length: rows t + n whose slots go on in this page
        int n = 1;
        for (int base = 1; offset + base < page_size; base += 32) {
            const int64_t r = t + base + lane;
            const bool goes_on = offset + base + lane < page_size && r < a.rows && a.slots[r] == slot + base + lane;
            const unsigned stop = ~__ballot_sync(0xffffffffu, goes_on);
            if (stop) {
                n = base + __ffs(stop) - 1;
                break;
            }
            n = base + 32;
        }
        const int64_t page = slot >> a.page_shift;
        const int vectors = n * per_row;
        // vector i of the run: row i / per_row (i < 2^15, exact in fp32)
        auto at = [&](int i, int& row, int& d) {
            row = static_cast<int>((static_cast<float>(i) + 0.5f) * inv_row);
            d = (i - row * per_row) * 8;
        };
        alignas(16) T kept[kKept][8];
        float most = 0.0f;
#pragma unroll
        for (int j = 0; j < kKept; ++j) {
            const int i = tid + j * kThreads;
            if (i < vectors) {
                int row, d;
                at(i, row, d);
                load8(x + (t + row) * token_stride + d, wide, kept[j]);
            }
        }
#pragma unroll
        for (int j = 0; j < kKept; ++j) {
            if (tid + j * kThreads < vectors) {
#pragma unroll
                for (int e = 0; e < 8; ++e) most = fmaxf(most, finite_size(to_f32(kept[j][e])));
            }
        }
        for (int i = tid + kKept * kThreads; i < vectors; i += kThreads) {
            int row, d;
            at(i, row, d);
            alignas(16) T v[8];
            load8(x + (t + row) * token_stride + d, wide, v);
#pragma unroll
            for (int e = 0; e < 8; ++e) most = fmaxf(most, finite_size(to_f32(v[e])));
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, d));
        __syncthreads();  // the run before is done with warp_max
        if (lane == 0) warp_max[warp] = most;
        float* const scale_at = a.scale[which] + page * a.heads + head;
        const float old = offset ? *scale_at : 0.0f;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kWarps; ++w) most = fmaxf(most, warp_max[w]);
        const float fresh = fmaxf(__fdiv_rn(most, kCodeMax), kLeastScale);
        const float scale = offset ? fmaxf(old, fresh) : fresh;
        const float inverse = __fdiv_rn(1.0f, scale);
        uint8_t* const tile = a.cache[which] + ((page * a.heads + head) << a.page_shift) * a.dim;
        if (offset && scale > old) {
            const float ratio = old * inverse;
            uint4* const held = reinterpret_cast<uint4*>(tile);
            for (int i = tid; i < offset * a.dim / 16; i += kThreads) {
                uint4 c = held[i];
                uint32_t* const w = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t u = w[k];
                    w[k] = code2(decode(u & 255u) * ratio, decode((u >> 8) & 255u) * ratio) |
                           (code2(decode((u >> 16) & 255u) * ratio, decode(u >> 24) * ratio) << 16);
                }
                held[i] = c;
            }
        }
        uint8_t* const to = tile + offset * a.dim;
#pragma unroll
        for (int j = 0; j < kKept; ++j) {
            const int i = tid + j * kThreads;
            if (i < vectors) *reinterpret_cast<uint2*>(to + i * 8) = encode8(kept[j], inverse);
        }
        for (int i = tid + kKept * kThreads; i < vectors; i += kThreads) {
            int row, d;
            at(i, row, d);
            alignas(16) T v[8];
            load8(x + (t + row) * token_stride + d, wide, v);
            *reinterpret_cast<uint2*>(to + i * 8) = encode8(v, inverse);
        }
        __syncthreads();  // every thread has read the page's old scale
        if (tid == 0) *scale_at = scale;
        t += n;
    }
}

template <typename T>
cudaError_t launch(const WriteArgs& a, cudaStream_t stream) {
    // rows that a block looks at; a run may go on behind them
    const int chunk = a.rows <= 4096 ? 1 : 32;
    bool wide[2];
    for (int i = 0; i < 2; ++i)
        wide[i] = ((reinterpret_cast<uintptr_t>(a.x[i]) | (a.token_stride[i] * sizeof(T)) |
                    (a.head_stride[i] * sizeof(T))) & 15) == 0;
    const dim3 grid(static_cast<unsigned>((a.rows + chunk - 1) / chunk), static_cast<unsigned>(a.heads), 2);
    cache_write_kernel<T><<<grid, kThreads, 0, stream>>>(a, chunk, wide[0], wide[1]);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_write(const WriteArgs& a, cudaStream_t stream) {
    if (a.dtype == kF32) return launch<float>(a, stream);
    if (a.dtype == kF16) return launch<__half>(a, stream);
    return launch<__nv_bfloat16>(a, stream);
}

}  // namespace lik
