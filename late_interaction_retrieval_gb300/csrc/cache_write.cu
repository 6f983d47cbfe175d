// cache_write.cu -- new keys and values into the 8-bit cache, one scale for
// each page and head.
//
// A run (rows of consecutive slots in one page) of one head has to be seen
// whole before its first value can be rounded: its largest value gives the
// page's scale.  A long run is a block's work and waits in shared memory
// between the two, read from memory once; what is on its way to shared memory
// takes no registers, so that a dozen blocks an SM keep enough of it under way.
// A short run (a decoded token, a few drafts) is a warp's, and is read again
// from L1.  The largest value is taken over the values' bits, two 16-bit ones
// at a time, which also shows whether any is not finite; only then each is
// looked at.
//
// What bounds it: issue slots (69%) as much as memory (60% of the DRAM's
// cycles): 15 instructions a value, of which the loops below have 6 or so (load,
// largest, product, half a conversion, store); the rest is what every block does
// for itself, a head and side at a time, to find the runs.  65521 rows of 8
// heads of 128, fp16: 80 us, 5.0 TB/s; fp32 126 us, 5.3 TB/s.  Values kept in registers instead of
// shared memory took 119 us, a persistent grid 130.
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "dtype_load.cuh"
#include "lik_internal.h"
#include "serve.h"

namespace lik {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int kShort = 128;        // vectors of 8 values of the longest run that is a warp's
constexpr int kMostStage = 32768;  // bytes of a run that wait in shared memory
constexpr int kMostChunk = 64;     // rows that a block looks at for runs that begin there
constexpr int kWords = (kMostChunk + 256) / 32;

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

__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

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
    __device__ __forceinline__ void load_shared(const T* p) {
        const uint4* const s = reinterpret_cast<const uint4*>(p);
#pragma unroll
        for (int i = 0; i < kWords / 4; ++i) {
            const uint4 v = s[i];
            w[4 * i] = v.x;
            w[4 * i + 1] = v.y;
            w[4 * i + 2] = v.z;
            w[4 * i + 3] = v.w;
        }
    }
    __device__ __forceinline__ float at(int i) const;
    // The largest of the sizes' bits so far and these; of 16-bit values two at
    // a time, each in its half of `most`.
    __device__ __forceinline__ uint32_t largest(uint32_t most) const {
#pragma unroll
        for (int i = 0; i < kWords; ++i)
            most = sizeof(T) == 4 ? max(most, w[i] & 0x7fffffffu) : max_halves(most, w[i] & 0x7fff7fffu);
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
    unsigned short h;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(y), "f"(x));
    return h;
}
// NaN for what is not finite (the conversion alone turns an infinity into the largest value).
__device__ __forceinline__ float nan_unless_finite(float x) { return is_finite(x) ? x : __int_as_float(0x7fffffff); }

__device__ __forceinline__ float decode(uint32_t code) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(code), __NV_E4M3)));
}

// 8 values in units of their scale, as codes.
template <bool kFinite, typename T>
__device__ __forceinline__ uint2 encode8(const Eight<T>& v, float inverse) {
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float x = v.at(2 * i), y = v.at(2 * i + 1);
        if (!kFinite) {
            x = nan_unless_finite(x);
            y = nan_unless_finite(y);
        }
        h[i] = code2(x * inverse, y * inverse);
    }
    return make_uint2(__byte_perm(h[0], h[1], 0x5410), __byte_perm(h[2], h[3], 0x5410));
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

__device__ __forceinline__ void copy16(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}

// One run of one head, by kGroup threads (a warp or the block) of which this
// is number `tid`.  stage: shared memory for `room` vectors (a block's), or 0.
template <typename T, int kGroup>
__device__ __forceinline__ void write_run(const Side<T>& a, const Run& r, int tid, uint32_t* of_warp, T* stage, int room) {
    const T* const x = a.x + r.row * a.token_stride;
    const int per_row = a.dim / 8, vectors = r.n * per_row;
    float* const scale_at = a.scale + r.page * a.heads + a.head;
    const float old = r.offset ? *scale_at : 0.0f;
    // The thread's vectors i = tid, tid + kGroup, ...: vector i lies in the run's row i / per_row.
    const int row0 = tid / per_row, d0 = tid - row0 * per_row, rows_on = kGroup / per_row, d_on = kGroup - rows_on * per_row;
    const int64_t on = rows_on * a.token_stride + d_on * 8, wrap = a.token_stride - a.dim;
    const bool staged = a.wide && vectors <= room;
    // body(vector of 8, its number)
    auto each = [&](auto body) {
        if (staged) {
#pragma unroll 2
            for (int i = tid; i < vectors; i += kGroup) {
                Eight<T> v;
                v.load_shared(stage + i * 8);
                body(v, i);
            }
            return;
        }
        const T* at = x + row0 * a.token_stride + d0 * 8;
        int d = d0;
#pragma unroll 2
        for (int i = tid; i < vectors; i += kGroup) {
            Eight<T> v;
            v.load(at, a.wide);
            body(v, i);
            d += d_on;
            at += on;
            if (d >= per_row) {
                d -= per_row;
                at += wrap;
            }
        }
    };
    if (staged) {  // a thread waits for what it fetched itself: it reads nothing else
        const T* at = x + row0 * a.token_stride + d0 * 8;
        int d = d0;
        uint32_t to = static_cast<uint32_t>(__cvta_generic_to_shared(stage + tid * 8));
#pragma unroll 4
        for (int i = tid; i < vectors; i += kGroup, to += kGroup * 8 * sizeof(T)) {
            copy16(to, at);
            if (sizeof(T) == 4) copy16(to + 16, at + 4);
            d += d_on;
            at += on;
            if (d >= per_row) {
                d -= per_row;
                at += wrap;
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
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
    uint32_t bits = 0;
    each([&](const Eight<T>& v, int) { bits = v.largest(bits); });
    bits = join(bits);
    const bool all_finite = bits < Bits<T>::kInf;
    if (!all_finite) {  // the largest of those that are finite
        bits = 0;
        each([&](const Eight<T>& v, int) {
#pragma unroll
            for (int e = 0; e < Eight<T>::kWords; ++e) {
                const uint32_t lo = sizeof(T) == 4 ? v.w[e] & 0x7fffffffu : v.w[e] & 0x7fffu;
                const uint32_t hi = sizeof(T) == 4 ? 0u : (v.w[e] >> 16) & 0x7fffu;
                bits = max(bits, lo < Bits<T>::kInf ? lo : 0u);
                bits = max(bits, hi < Bits<T>::kInf ? hi : 0u);
            }
        });
        bits = join(bits);
    }
    const float fresh = fmaxf(__fdiv_rn(size_of_bits<T>(bits), kCodeMax), kLeastScale);
    const float scale = r.offset ? fmaxf(old, fresh) : fresh;
    const float inverse = __fdiv_rn(1.0f, scale);
    uint8_t* const tile = a.cache + ((r.page * a.heads + a.head) << a.page_shift) * a.dim;
    if (r.offset && scale > old) {
        const float ratio = old * inverse;
        uint4* const held = reinterpret_cast<uint4*>(tile);
#pragma unroll 1
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
    uint2* const to = reinterpret_cast<uint2*>(tile + r.offset * a.dim);
    if (all_finite) each([&](const Eight<T>& v, int i) { to[i] = encode8<true>(v, inverse); });
    else each([&](const Eight<T>& v, int i) { to[i] = encode8<false>(v, inverse); });
    __syncwarp();  // every lane has read the old scale (every warp has: it did before the join)
    if (tid == 0) *scale_at = scale;
}

// Blocks are (chunk, keys or values, head), heads next to one another: blocks that run together read whole rows and
// write whole pages.
template <typename T>
__global__ void __launch_bounds__(kThreads) cache_write_kernel(const WriteArgs a, int chunk, int room, bool wide_k, bool wide_v) {
    extern __shared__ __align__(16) uint8_t stage[];
    __shared__ uint32_t of_warp[kWarps];
    __shared__ unsigned on_of[kWords], begins_of[kMostChunk / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int head = static_cast<int>(blockIdx.x % a.heads), which = blockIdx.y;
    const int64_t t0 = static_cast<int64_t>(blockIdx.x / a.heads) * chunk;
    const int page_size = 1 << a.page_shift, words = (chunk + page_size + 31) / 32;
    // Rows t0, t0 + 1, ...: those of the chunk, and as many behind it as a run that begins there may have.  Bit l of
    // word k: row t0 + 32 k + l goes on with the run of the row before; a run begins there.
    const int64_t n_slots = a.pages << a.page_shift;
    for (int k = warp; k < words; k += kWarps) {
        const int64_t r = t0 + 32 * k + lane;
        const int64_t slot = r < a.rows ? a.slots[r] : -1, before = r < a.rows && r > 0 ? a.slots[r - 1] : -1;
        const bool valid = slot >= 0 && slot < n_slots;
        const bool goes_on = valid && (slot & (page_size - 1)) != 0 && before >= 0 && before + 1 == slot;
        const unsigned on = __ballot_sync(0xffffffffu, goes_on);
        const unsigned begins = __ballot_sync(0xffffffffu, valid && !goes_on && 32 * k + lane < chunk);
        if (lane == 0) {
            on_of[k] = on;
            if (k < kMostChunk / 32) begins_of[k] = begins;
        }
    }
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
    const int short_rows = kShort / (a.dim / 8);
    int shorts = 0;
    __syncthreads();
#pragma unroll 1
    for (int k = 0; k < kMostChunk / 32 && 32 * k < chunk; ++k) {
#pragma unroll 1
        for (unsigned rest = begins_of[k]; rest; rest &= rest - 1) {
            const int l = __ffs(rest) - 1;
            Run r;
            r.row = t0 + 32 * k + l;
            const int64_t slot = a.slots[r.row];
            r.page = slot >> a.page_shift;
            r.offset = static_cast<int>(slot & (page_size - 1));
            // rows behind it that go on: the run ends in its page, so within the words
            const unsigned off = l == 31 ? 0u : ~on_of[k] >> (l + 1);
            r.n = 1 + (off ? min(__ffs(off) - 1, 31 - l) : 31 - l);
            for (int j = k + 1; r.n == 32 * (j - k) - l && j < words; ++j)
                r.n += on_of[j] == 0xffffffffu ? 32 : __ffs(~on_of[j]) - 1;
            if (r.n <= short_rows) {
                if (shorts++ % kWarps == warp) write_run<T, 32>(side, r, lane, of_warp, nullptr, 0);
            } else {
                write_run<T, kThreads>(side, r, tid, of_warp, reinterpret_cast<T*>(stage), room);
            }
        }
    }
}

template <typename T>
cudaError_t launch(const WriteArgs& a, cudaStream_t stream) {
    // rows that a block looks at; a run may go on behind them
    const int chunk = a.rows <= 512 ? 1 : (a.rows <= 8192 ? 8 : kMostChunk);
    bool wide[2];
    for (int i = 0; i < 2; ++i)
        wide[i] = ((reinterpret_cast<uintptr_t>(a.x[i]) | (a.token_stride[i] * sizeof(T)) |
                    (a.head_stride[i] * sizeof(T))) & 15) == 0;
    // shared memory for the longest run there can be, or kMostStage of it; longer runs are read twice
    const int64_t most = a.rows, page = int64_t(1) << a.page_shift;
    const int64_t longest = (most < page ? most : page) * (a.dim / 8), space = kMostStage / (8 * sizeof(T));
    const int room = static_cast<int>(longest < space ? longest : space);
    const int64_t blocks = (a.rows + chunk - 1) / chunk * a.heads;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    cache_write_kernel<T><<<dim3(static_cast<unsigned>(blocks), 2), kThreads, room * 8 * sizeof(T), stream>>>(
        a, chunk, room, wide[0], wide[1]);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_write(const WriteArgs& a, cudaStream_t stream) {
    if (a.dtype == kF32) return launch<float>(a, stream);
    if (a.dtype == kF16) return launch<__half>(a, stream);
    return launch<__nv_bfloat16>(a, stream);
}

}  // namespace lik
