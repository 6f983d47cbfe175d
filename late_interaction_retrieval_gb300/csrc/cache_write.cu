// cache_write.cu -- new keys and values into the 8-bit cache, one scale for
// each page and head.
//
// A run (rows of consecutive slots in one page) of one head has to be seen
// whole before its first value can be rounded: its largest value gives the
// page's scale.  It is kept in registers between the two, so that it is read
// once: a long run by a block, a short one (a decoded token, a few drafts) by
// a warp of it.  The largest value is taken over the values' bits, two 16-bit
// ones at a time, which also shows whether any is not finite; only then each
// is looked at.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "dtype_load.cuh"
#include "lik_internal.h"
#include "serve.h"

namespace lik {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kKept = 8;         // vectors of 8 values that a thread of a block keeps
constexpr int kKeptByWarp = 2;   // of a warp; longer runs are a block's

template <typename T>
struct Bits;
template <>
struct Bits<float> {
    static constexpr uint32_t kInf = 0x7f800000u;
};
template <>
struct Bits<__half> {
    static constexpr uint32_t kInf = 0x7c00u;
};
template <>
struct Bits<__nv_bfloat16> {
    static constexpr uint32_t kInf = 0x7f80u;
};

// 8 values as they lie in memory.
template <typename T>
struct Eight {
    static constexpr int kWords = sizeof(T) * 2;
    uint32_t w[kWords];

    __device__ __forceinline__ void load(const T* p, bool wide) {
        if (wide) {
            const uint4* const s = reinterpret_cast<const uint4*>(p);
#pragma unroll
            for (int i = 0; i < kWords / 4; ++i) {
                const uint4 v = __ldg(s + i);
                w[4 * i] = v.x;
                w[4 * i + 1] = v.y;
                w[4 * i + 2] = v.z;
                w[4 * i + 3] = v.w;
            }
        } else if (sizeof(T) == 4) {
            const uint32_t* const s = reinterpret_cast<const uint32_t*>(p);
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[i] = s[i];
        } else {
            const uint16_t* const s = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
            for (int i = 0; i < kWords; ++i) w[i] = s[2 * i] | (static_cast<uint32_t>(s[2 * i + 1]) << 16);
        }
    }
    __device__ __forceinline__ float at(int i) const;
    // The largest of the sizes' bits so far and these; of 16-bit values two at
    // a time, each in its half of `most`.
    __device__ __forceinline__ uint32_t largest(uint32_t most) const {
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            most = sizeof(T) == 4 ? max(most, w[i] & 0x7fffffffu) : __vmaxu2(most, w[i] & 0x7fff7fffu);
        return most;
    }
};
template <>
__device__ __forceinline__ float Eight<float>::at(int i) const {
    return __uint_as_float(w[i]);
}
template <>
__device__ __forceinline__ float Eight<__half>::at(int i) const {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(w[i / 2] >> (16 * (i & 1)))));
}
template <>
__device__ __forceinline__ float Eight<__nv_bfloat16>::at(int i) const {
    return __uint_as_float(i & 1 ? w[i / 2] & 0xffff0000u : w[i / 2] << 16);
}

template <typename T>
__device__ __forceinline__ float size_of_bits(uint32_t b);
template <>
__device__ __forceinline__ float size_of_bits<float>(uint32_t b) {
    return __uint_as_float(b);
}
template <>
__device__ __forceinline__ float size_of_bits<__half>(uint32_t b) {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(b)));
}
template <>
__device__ __forceinline__ float size_of_bits<__nv_bfloat16>(uint32_t b) {
    return __uint_as_float(b << 16);
}

__device__ __forceinline__ bool is_finite(float x) { return fabsf(x) <= 3.402823466e38f; }

__device__ __forceinline__ uint32_t code2(float x, float y) {
    return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}
// NaN for what is not finite (the conversion alone turns an infinity into the largest value).
__device__ __forceinline__ float nan_unless_finite(float x) { return is_finite(x) ? x : __int_as_float(0x7fffffff); }

__device__ __forceinline__ float decode(uint32_t code) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3)));
}

// 8 values in units of their scale, as codes.
template <typename T>
__device__ __forceinline__ uint2 encode8(const Eight<T>& v, float inverse, bool all_finite) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float x = v.at(2 * i), y = v.at(2 * i + 1);
        if (!all_finite) {
            x = nan_unless_finite(x);
            y = nan_unless_finite(y);
        }
        h[i] = code2(x * inverse, y * inverse);
    }
    return make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
}

// Keys or values.
template <typename T>
struct Side {
    const T* x;  // of the block's head
    int64_t token_stride;
    uint8_t* cache;
    float* scale;
    int heads, head, dim, page_shift;
    bool wide;
};

struct Run {
    int64_t row;  // its first row
    int64_t page;
    int offset, n;
};

// One run of one head, by kGroup threads (a warp or the block) of which this
// is number `tid`.
template <typename T, int kGroup, int kHeld>
__device__ __forceinline__ void write_run(const Side<T>& a, const Run& r, int tid, uint32_t* of_warp) {
    const T* const x = a.x + r.row * a.token_stride;
    const int64_t token_stride = a.token_stride;
    const bool wide = a.wide;
    const int per_row = a.dim / 8, vectors = r.n * per_row;
    const float inv_row = 1.0f / static_cast<float>(per_row);
    float* const scale_at = a.scale + r.page * a.heads + a.head;
    const float old = r.offset ? *scale_at : 0.0f;
    // vector i of the run lies in its row i / per_row (i < 2^12, exact in fp32)
    auto from = [&](int i) {
        const int row = static_cast<int>((static_cast<float>(i) + 0.5f) * inv_row);
        return x + row * token_stride + (i - row * per_row) * 8;
    };
    Eight<T> kept[kHeld];
    uint32_t bits = 0;
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
        if (tid + j * kGroup < vectors) kept[j].load(from(tid + j * kGroup), wide);
#pragma unroll
    for (int j = 0; j < kHeld; ++j)
        if (tid + j * kGroup < vectors) bits = kept[j].largest(bits);
    for (int i = tid + kHeld * kGroup; i < vectors; i += kGroup) {
        Eight<T> v;
        v.load(from(i), wide);
        bits = v.largest(bits);
    }
    auto join = [&](uint32_t b) {
        if (sizeof(T) == 2) b = max(b & 0xffffu, b >> 16);
        b = __reduce_max_sync(0xffffffffu, b);
        if (kGroup > 32) {
            __syncthreads();  // of_warp is free
            if ((tid & 31) == 0) of_warp[tid >> 5] = b;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < kWarps; ++w) b = max(b, of_warp[w]);
        }
        return b;
    };
    bits = join(bits);
    const bool all_finite = bits < Bits<T>::kInf;
    if (!all_finite) {  // the largest of those that are finite
        bits = 0;
        for (int i = tid; i < vectors; i += kGroup) {
            Eight<T> v;
            v.load(from(i), wide);
#pragma unroll
            for (int e = 0; e < Eight<T>::kWords; ++e) {
                const uint32_t lo = sizeof(T) == 4 ? v.w[e] & 0x7fffffffu : v.w[e] & 0x7fffu;
                const uint32_t hi = sizeof(T) == 4 ? 0u : (v.w[e] >> 16) & 0x7fffu;
                bits = max(bits, lo < Bits<T>::kInf ? lo : 0u);
                bits = max(bits, hi < Bits<T>::kInf ? hi : 0u);
            }
        }
        bits = join(bits);
    }
    const float fresh = fmaxf(__fdiv_rn(size_of_bits<T>(bits), kCodeMax), kLeastScale);
    const float scale = r.offset ? fmaxf(old, fresh) : fresh;
    const float inverse = __fdiv_rn(1.0f, scale);
    uint8_t* const tile = a.cache + ((r.page * a.heads + a.head) << a.page_shift) * a.dim;
    if (r.offset && scale > old) {
        const float ratio = old * inverse;
        uint4* const held = reinterpret_cast<uint4*>(tile);
        for (int i = tid; i < r.offset * a.dim / 16; i += kGroup) {
            uint4 c = held[i];
            uint32_t* const w = reinterpret_cast<uint32_t*>(&c);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const uint32_t u = w[k];
                w[k] = code2(nan_unless_finite(decode(u & 255u) * ratio), nan_unless_finite(decode((u >> 8) & 255u) * ratio)) |
                       (code2(nan_unless_finite(decode((u >> 16) & 255u) * ratio), nan_unless_finite(decode(u >> 24) * ratio))
                        << 16);
            }
            held[i] = c;
        }
    }
    uint8_t* const to = tile + r.offset * a.dim;
#pragma unroll
    for (int j = 0; j < kHeld; ++j) {
        const int i = tid + j * kGroup;
        if (i < vectors) *reinterpret_cast<uint2*>(to + i * 8) = encode8(kept[j], inverse, all_finite);
    }
    for (int i = tid + kHeld * kGroup; i < vectors; i += kGroup) {
        Eight<T> v;
        v.load(from(i), wide);
        *reinterpret_cast<uint2*>(to + i * 8) = encode8(v, inverse, all_finite);
    }
    __syncwarp();  // every lane has read the old scale (every warp has: it did before the join)
    if (tid == 0) *scale_at = scale;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const WriteArgs a, int chunk, bool wide_k, bool wide_v) {
    __shared__ uint32_t of_warp[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int head = blockIdx.y, which = blockIdx.z;
    Side<T> side;
    side.x = static_cast<const T*>(which ? a.x[1] : a.x[0]) + head * (which ? a.head_stride[1] : a.head_stride[0]);
    side.token_stride = which ? a.token_stride[1] : a.token_stride[0];
    side.cache = which ? a.cache[1] : a.cache[0];
    side.scale = which ? a.scale[1] : a.scale[0];
    side.heads = a.heads;
    side.head = head;
    side.dim = a.dim;
    side.page_shift = a.page_shift;
    side.wide = which ? wide_v : wide_k;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x) * chunk;
    const int page_size = 1 << a.page_shift;
    const int64_t n_slots = a.pages << a.page_shift;

    // lane l looks at row t0 + l: does a run begin there, and if not, does one go on?
    const int64_t t = t0 + lane;
    const bool looked = lane < chunk && t < a.rows;
    const int64_t slot = looked ? a.slots[t] : -1;
    const int64_t before = looked && t > 0 ? a.slots[t - 1] : -1;
    const bool valid = slot >= 0 && slot < n_slots;
    const int offset = static_cast<int>(slot & (page_size - 1));
    const bool goes_on = valid && offset != 0 && before >= 0 && before + 1 == slot;
    const unsigned begins = __ballot_sync(0xffffffffu, valid && !goes_on);
    const unsigned on = __ballot_sync(0xffffffffu, goes_on);

    const int short_rows = kKeptByWarp * 32 / (a.dim / 8);  // of a run that a warp keeps
    int number = 0;
    for (unsigned rest = begins; rest; rest &= rest - 1) {
        const int l = __ffs(rest) - 1;
        Run r;
        r.row = t0 + l;
        const int64_t s = __shfl_sync(0xffffffffu, slot, l);
        r.page = s >> a.page_shift;
        r.offset = static_cast<int>(s & (page_size - 1));
        // rows of the chunk behind it that go on; the run may pass the chunk
        const unsigned behind = l == 31 ? 0u : ~(on >> (l + 1));
        const int in_chunk = chunk - 1 - l;
        int n = l == 31 ? 0 : (behind ? __ffs(behind) - 1 : 31);
        n = n < in_chunk ? n : in_chunk;
        if (n == in_chunk) {
            for (int base = n + 1; r.offset + base < page_size; base += 32) {
                const int64_t k = r.row + base + lane;
                const bool more = r.offset + base + lane < page_size && k < a.rows && a.slots[k] == s + base + lane;
                const unsigned stop = ~__ballot_sync(0xffffffffu, more);
                n = base - 1 + (stop ? __ffs(stop) - 1 : 32);
                if (stop) break;
            }
        }
        r.n = n + 1;
        if (r.n <= short_rows) {
            if (number++ % kWarps == warp) write_run<T, 32, kKeptByWarp>(side, r, lane, of_warp);
        } else {
            write_run<T, kThreads, kKept>(side, r, tid, of_warp);
        }
    }
}

template <typename T>
cudaError_t launch(const WriteArgs& a, cudaStream_t stream) {
    // rows that a block looks at; a run may go on behind them
    const int chunk = a.rows <= 512 ? 1 : (a.rows <= 8192 ? 8 : 32);
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
