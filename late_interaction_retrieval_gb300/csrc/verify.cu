// verify.cu -- drafted tokens against the target's probabilities.
//
// First launch: every row's largest logit and sum of exponentials, a row cut
// into parts over blocks (a handful of rows has to fill the chip).  Second
// launch: each block of a request joins its rows' parts, finds the first
// draft that does not pass, and races its share of that row's columns against
// the noise; the last block of a request to finish writes its tokens.
//
// What bounds them: the first reads every logit once at 66% of the DRAM's
// cycles, its issue slots 72% used (an exponential a logit); the second reads
// a row of either model and the noise for each request.  64 requests of 4
// drafts, 128000 columns, bf16: 48 us, 29 and 23 with cold caches; what the
// second launch does before it needs the first's results overlaps its end.
#include <cuda_runtime.h>

#include "dtype_load.cuh"
#include "lik_internal.h"
#include "serve.h"

namespace lik {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxParts = 64;
constexpr float kLn2 = 0.693147180559945309f;

struct Plan {
    int parts;        // of a row in the first launch
    int64_t part;     // columns of a part
    int races;        // blocks of a request in the second
    int64_t share;    // columns of one
    float2* stats;    // [rows, parts]: largest logit, sum of exponentials
    unsigned long long* best;  // [requests]: the race's key, ~column
    unsigned int* done;        // [requests]: blocks that have finished
};

// exp(scale * d), d <= 0, to about 2^-22: the product's rounding is put right.
struct Scale {
    float hi, lo;  // scale * log2(e) in two parts
};
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float exp_scaled(float d, Scale c) {
    const float t = d * c.hi;
    const float rest = fmaf(d, c.lo, fmaf(d, c.hi, -t));
    const float e = exp2_fast(t);
    // below every fp32 value the product may have overflowed, and `rest` with it
    return t < -200.0f ? 0.0f : fmaf(e, rest * kLn2, e);
}

__device__ __forceinline__ float2 join(float2 x, float2 y, Scale c) {
    // the largest is taken without NaN, which stays in the sum: a side's sum is 0 only if it has nothing
    const float m = fmaxf(x.x, y.x);
    const float base = m == -INFINITY ? 0.0f : m;
    const float sx = x.y == 0.0f ? 0.0f : x.y * exp_scaled(x.x - base, c);
    const float sy = y.y == 0.0f ? 0.0f : y.y * exp_scaled(y.x - base, c);
    return make_float2(m, sx + sy);
}

__device__ __forceinline__ float2 warp_join(float2 v, Scale c) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const float2 o = make_float2(__shfl_xor_sync(0xffffffffu, v.x, d), __shfl_xor_sync(0xffffffffu, v.y, d));
        v = join(v, o, c);
    }
    return v;
}

// 16 bytes of logits, widened.
template <typename T>
struct Vec {
    static constexpr int n = 16 / sizeof(T);
    uint4 raw;
    __device__ __forceinline__ void load(const T* p) { raw = __ldg(reinterpret_cast<const uint4*>(p)); }
    // The largest (a NaN is passed over): of 16-bit logits two at a time, before they are widened.
    __device__ __forceinline__ float largest() const;
    __device__ __forceinline__ void widen(float (&f)[n]) const {
        const T* const e = reinterpret_cast<const T*>(&raw);
#pragma unroll
        for (int i = 0; i < n; ++i) f[i] = to_f32(e[i]);
    }
};

template <>
__device__ __forceinline__ float Vec<float>::largest() const {
    return fmaxf(fmaxf(__uint_as_float(raw.x), __uint_as_float(raw.y)), fmaxf(__uint_as_float(raw.z), __uint_as_float(raw.w)));
}
template <>
__device__ __forceinline__ float Vec<__half>::largest() const {
    const __half2* const h = reinterpret_cast<const __half2*>(&raw);
    const __half2 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
}
template <>
__device__ __forceinline__ float Vec<__nv_bfloat16>::largest() const {
    const __nv_bfloat162* const h = reinterpret_cast<const __nv_bfloat162*>(&raw);
    const __nv_bfloat162 m = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
    return fmaxf(__low2float(m), __high2float(m));
}

// Two fp32 numbers in one register pair, for one instruction on both.
__device__ __forceinline__ uint64_t both(float x, float y) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(x), "f"(y));
    return d;
}
__device__ __forceinline__ float2 each_of(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t add_both(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t mul_both(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// One logit's (largest, sum): nothing for -inf, a NaN sum for NaN.
__device__ __forceinline__ float2 one(float z) {
    return make_float2(z, z == -INFINITY ? 0.0f : (z == z ? 1.0f : z));
}

template <typename T>
__global__ void __launch_bounds__(kThreads) verify_stats(const VerifyArgs a, const Plan w, Scale c) {
    __shared__ float2 of_warp[kWarps];
    constexpr int kVec = Vec<T>::n, kUnroll = 32 / kVec;  // 32 columns a thread and turn
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x;
    const int64_t targets = a.drafts + a.requests;
    const T* const z = row < targets ? static_cast<const T*>(a.target) + row * a.target_stride
                                     : static_cast<const T*>(a.draft) + (row - targets) * a.draft_stride;
    if (blockIdx.y == 0 && row < a.requests && tid == 0) {
        w.best[row] = 0;
        w.done[row] = 0;
    }
    const int64_t c0 = blockIdx.y * w.part, c1 = c0 + w.part < a.cols ? c0 + w.part : a.cols;
    float2 v = make_float2(-INFINITY, 0.0f);
    if (c0 < c1) {
        // columns up to the first 16-byte boundary and behind the last one alone
        const int64_t to_wide = ((16 - (reinterpret_cast<uintptr_t>(z + c0) & 15)) & 15) / sizeof(T);
        const int64_t head = to_wide < c1 - c0 ? to_wide : c1 - c0;
        const int64_t vecs = (c1 - c0 - head) / kVec, tail = c0 + head + vecs * kVec;
        if (tid < head) v = join(v, one(load_f32(z + c0 + tid)), c);
        if (tid < c1 - tail) v = join(v, one(load_f32(z + tail + tid)), c);
        const T* const wide = z + c0 + head;
        // the next turn's loads are on their way while this one's exponentials are taken
        Vec<T> x[kUnroll];
        auto fetch = [&](int64_t i) {
#pragma unroll
            for (int u = 0; u < kUnroll; ++u)
                if (i + u * kThreads < vecs) x[u].load(wide + (i + u * kThreads) * kVec);
        };
        fetch(tid);
        for (int64_t i = tid; i < vecs; i += kUnroll * kThreads) {
            Vec<T> now[kUnroll];
            float m = v.x;
            int have = 0;  // of the turn's vectors
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                now[u] = x[u];
                if (i + u * kThreads < vecs) {
                    m = fmaxf(m, now[u].largest());
                    have = u + 1;
                }
            }
            fetch(i + kUnroll * kThreads);
            // All of it -inf so far: 0 stands in, and every term is 0.  A NaN makes its own term one.  The maximum is
            // subtracted before the product with the scale, two logits an instruction: no difference is above 0 and the
            // largest is 0 whatever the logits' size and the scale, which a product rounded first would not give.
            const float base = m == -INFINITY ? 0.0f : m;
            const uint64_t minus = both(-base, -base), factor = both(c.hi, c.hi);
            uint64_t s[2] = {0, 0};
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (u >= have) continue;
                float f[kVec];
                now[u].widen(f);
#pragma unroll
                for (int e = 0; e < kVec; e += 2) {
                    const float2 t = each_of(mul_both(add_both(both(f[e], f[e + 1]), minus), factor));
                    s[(e >> 1) & 1] = add_both(s[(e >> 1) & 1], both(exp2_fast(t.x), exp2_fast(t.y)));
                }
            }
            const float2 sum = each_of(add_both(s[0], s[1]));
            const float kept = v.y == 0.0f ? 0.0f : v.y * exp_scaled(v.x - base, c);
            v = make_float2(m, kept + (sum.x + sum.y));
        }
    }
    v = warp_join(v, c);
    if (lane == 0) of_warp[warp] = v;
    __syncthreads();
    if (tid == 0) {
        for (int i = 1; i < kWarps; ++i) v = join(v, of_warp[i], c);
        w.stats[row * w.parts + blockIdx.y] = v;
    }
}

// A row's statistics from its parts, by a whole warp.
__device__ __forceinline__ float2 row_stats(const Plan& w, int64_t row, Scale c) {
    const int lane = threadIdx.x & 31;
    float2 v = make_float2(-INFINITY, 0.0f);
    for (int i = lane; i < w.parts; i += 32) v = join(v, w.stats[row * w.parts + i], c);
    return warp_join(v, c);
}

// The sum is 0 only for a row without any mass; a NaN or +inf logit leaves a
// NaN, which fails every comparison below.
__device__ __forceinline__ float prob(float z, float2 s, Scale c) {
    return s.y == 0.0f ? 0.0f : exp_scaled(z - s.x, c) / s.y;
}

// A thread's best column: the largest quotient above 0, the first of equals.
struct Best {
    float key = 0.0f;
    int64_t col = 0;
    __device__ __forceinline__ void offer(float r, float noise, int64_t k) {
        const float q = __fdividef(r, noise);
        if (q > key) {
            key = q;
            col = k;
        }
    }
    __device__ __forceinline__ unsigned long long packed() const {
        if (!(key > 0.0f)) return 0;
        return (static_cast<unsigned long long>(__float_as_uint(key)) << 32) | (0xffffffffu - static_cast<unsigned>(col));
    }
};

__device__ __forceinline__ unsigned long long block_max(unsigned long long v, unsigned long long* of_warp) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const unsigned long long o = __shfl_xor_sync(0xffffffffu, v, d);
        v = o > v ? o : v;
    }
    if ((threadIdx.x & 31) == 0) of_warp[threadIdx.x >> 5] = v;
    __syncthreads();
    for (int i = 0; i < kWarps; ++i) v = of_warp[i] > v ? of_warp[i] : v;
    __syncthreads();
    return v;
}

// Drafts whose rows' statistics a block keeps.
constexpr int kKept = 64;

template <typename T>
__global__ void __launch_bounds__(kThreads) verify_draw(const VerifyArgs a, const Plan w, Scale c, bool wide) {
    __shared__ unsigned long long of_warp[kWarps];
    __shared__ int first_fail, is_last;
    __shared__ float2 stat_p[kKept], stat_q[kKept];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, b = blockIdx.y;
    const int64_t targets = a.drafts + a.requests;
    int64_t lo = a.offsets[b], hi = a.offsets[b + 1];
    lo = lo < 0 ? 0 : (lo < a.drafts ? lo : a.drafts);
    hi = hi < lo ? lo : (hi < a.drafts ? hi : a.drafts);
    const int n = static_cast<int>(hi - lo);
    const T* const target = static_cast<const T*>(a.target);
    const T* const draft = static_cast<const T*>(a.draft);
    const bool writes = blockIdx.x == 0;  // the tokens that pass; the drawn one is the last block's
    if (tid == 0) first_fail = n;
    __syncthreads();
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // a warp takes a draft at a time, and the row behind the last (which always "passes")
    for (int i = warp; i <= n; i += kWarps) {
        // one lane's view of what other warps write, so that the warp stays whole
        if (__shfl_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&first_fail), 0) < i) break;
        const int64_t row = lo + i, tr = row + b;
        const int x = i < n ? a.drafted[row] : -1;
        const float u = i < n ? a.uniform[row] : 0.0f;
        const bool inside = x >= 0 && x < a.cols;
        const float zp = inside ? load_f32(target + tr * a.target_stride + x) : 0.0f;
        const float zq = inside && draft ? load_f32(draft + row * a.draft_stride + x) : 0.0f;
        const float2 sp = row_stats(w, tr, c);
        const float2 sq = i < n && draft ? row_stats(w, targets + row, c) : make_float2(0.0f, 0.0f);
        if (lane == 0) {
            if (i < kKept) {
                stat_p[i] = sp;
                stat_q[i] = sq;
            }
            // a draft row without mass is no distribution: as with a NaN in it, its draft does not pass
            const float p = prob(zp, sp, c), q = !draft ? 1.0f : sq.y == 0.0f ? NAN : prob(zq, sq, c);
            if (i < n && !(inside && static_cast<double>(u) * q < static_cast<double>(p))) atomicMin(&first_fail, i);
            if (writes && i < n) {
                a.tokens[tr] = x;
                a.logp[tr] = a.scale * (zp - sp.x) - logf(sp.y);
            }
        }
    }
    __syncthreads();
    const int kept = first_fail;
    const int64_t tr = lo + b + kept, dr = lo + kept;
    const bool residual = kept < n;
    if (writes) {  // behind what passed there is nothing (but the token that is drawn)
        for (int i = kept + 1 + tid; i <= n; i += kThreads) {
            a.tokens[lo + b + i] = -1;
            a.logp[lo + b + i] = 0.0f;
        }
        if (tid == 0) a.accepted[b] = kept;
        if (b == a.requests - 1) {  // rows behind the last request's
            for (int64_t r = hi + b + 1 + tid; r < targets; r += kThreads) {
                a.tokens[r] = -1;
                a.logp[r] = 0.0f;
            }
        }
    }
    float2 sp, sq;
    if (kept < kKept) {
        sp = stat_p[kept];
        sq = stat_q[kept];
    } else {
        sp = row_stats(w, tr, c);
        sq = residual && draft ? row_stats(w, targets + dr, c) : make_float2(0.0f, 0.0f);
    }
    const T* const z = target + tr * a.target_stride;
    const T* const y = residual && draft ? draft + dr * a.draft_stride : nullptr;
    const int64_t struck = residual && !draft ? a.drafted[dr] : -1;
    const float* const noise = a.noise + b * a.cols;
    const int64_t c0 = blockIdx.x * w.share, c1 = c0 + w.share < a.cols ? c0 + w.share : a.cols;
    // probabilities by the sums' reciprocals
    const float ip = sp.y == 0.0f ? 0.0f : 1.0f / sp.y, iq = !y || sq.y == 0.0f ? 0.0f : 1.0f / sq.y;
    auto left_of = [&](float zp, float zq, int64_t k) {
        float r = exp_scaled(zp - sp.x, c) * ip;
        if (y) r = fmaxf(r - exp_scaled(zq - sq.x, c) * iq, 0.0f);
        return k == struck ? 0.0f : r;
    };
    Best mine;
    if (wide) {
        constexpr int kVec = Vec<T>::n, kTurn = 16 / kVec;  // 16 columns a thread and turn
        for (int64_t k0 = c0 + tid * kVec; k0 < c1; k0 += kThreads * kVec * kTurn) {
            Vec<T> xp[kTurn], xq[kTurn];
            float4 e[kTurn][kVec / 4];
#pragma unroll
            for (int t = 0; t < kTurn; ++t) {
                const int64_t k = k0 + t * kThreads * kVec;
                if (k < c1) {
                    xp[t].load(z + k);
                    if (y) xq[t].load(y + k);
                    else xq[t].raw = make_uint4(0, 0, 0, 0);
#pragma unroll
                    for (int i = 0; i < kVec / 4; ++i) e[t][i] = __ldg(reinterpret_cast<const float4*>(noise + k) + i);
                }
            }
#pragma unroll
            for (int t = 0; t < kTurn; ++t) {
                const int64_t k = k0 + t * kThreads * kVec;
                if (k < c1) {
                    float fp[kVec], fq[kVec];
                    xp[t].widen(fp);
                    xq[t].widen(fq);
#pragma unroll
                    for (int i = 0; i < kVec; ++i)
                        mine.offer(left_of(fp[i], fq[i], k + i), reinterpret_cast<const float*>(e[t])[i], k + i);
                }
            }
        }
    } else {
        constexpr int kTurn = 8;
        for (int64_t k0 = c0 + tid; k0 < c1; k0 += kThreads * kTurn) {
            float fp[kTurn], fq[kTurn], e[kTurn];
#pragma unroll
            for (int t = 0; t < kTurn; ++t) {
                const int64_t k = k0 + t * kThreads;
                fp[t] = k < c1 ? load_f32(z + k) : -INFINITY;
                fq[t] = y && k < c1 ? load_f32(y + k) : 0.0f;
                e[t] = k < c1 ? __ldg(noise + k) : INFINITY;
            }
#pragma unroll
            for (int t = 0; t < kTurn; ++t) mine.offer(left_of(fp[t], fq[t], k0 + t * kThreads), e[t], k0 + t * kThreads);
        }
    }
    unsigned long long best = block_max(mine.packed(), of_warp);
    if (tid == 0) {
        if (best) atomicMax(w.best + b, best);
        __threadfence();
        is_last = atomicAdd(w.done + b, 1u) + 1 == gridDim.x;
        __threadfence();
    }
    __syncthreads();
    if (!is_last) return;
    best = *reinterpret_cast<volatile unsigned long long*>(w.best + b);
    if (best == 0 && residual) {  // nothing is left of the target over the draft: the target itself
        Best all;
        for (int64_t k = tid; k < a.cols; k += kThreads) all.offer(exp_scaled(load_f32(z + k) - sp.x, c) * ip, noise[k], k);
        best = block_max(all.packed(), of_warp);
    }
    if (tid == 0) {
        const int token = best ? static_cast<int>(0xffffffffu - static_cast<unsigned>(best)) : -1;
        a.tokens[tr] = token;
        // in natural logarithms: scale * (z - max) - log(sum)
        a.logp[tr] = token >= 0 ? a.scale * (load_f32(z + token) - sp.x) - logf(sp.y) : 0.0f;
    }
}

// Parts of each of `rows` rows: as many as fill the chip once, of 4096 columns
// at least.
int parts_of(int64_t rows, int64_t cols, int64_t blocks) {
    int64_t p = blocks / (rows > 0 ? rows : 1);
    const int64_t most = (cols + 4095) / 4096;
    p = p < most ? p : most;
    return static_cast<int>(p < 1 ? 1 : (p < kMaxParts ? p : kMaxParts));
}

size_t round16(size_t n) { return (n + 15) & ~static_cast<size_t>(15); }

template <typename T>
cudaError_t launch(const VerifyArgs& a, const Plan& w, Scale c, cudaStream_t stream) {
    const int64_t rows = a.drafts + a.requests + (a.draft ? a.drafts : 0);
    verify_stats<T><<<dim3(static_cast<unsigned>(rows), w.parts), kThreads, 0, stream>>>(a, w, c);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    // 16-byte loads from all three rows: every row of each starts on a 16-byte boundary
    auto whole = [](const void* p, int64_t stride, size_t size) {
        return ((reinterpret_cast<uintptr_t>(p) | (static_cast<uintptr_t>(stride) * size)) & 15) == 0;
    };
    const bool wide = a.cols % Vec<T>::n == 0 && whole(a.target, a.target_stride, sizeof(T)) &&
                      whole(a.noise, a.cols, 4) && (!a.draft || whole(a.draft, a.draft_stride, sizeof(T)));
    // its blocks are in place when the first launch ends
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(w.races, a.requests);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, verify_draw<T>, a, w, c, wide);
}

}  // namespace

size_t verify_workspace(int64_t drafts, int64_t requests, int64_t) {
    return round16(sizeof(float2) * kMaxParts * static_cast<size_t>(2 * drafts + requests)) +
           round16(sizeof(unsigned long long) * requests) + round16(sizeof(unsigned int) * requests);
}

cudaError_t launch_verify(const VerifyArgs& a, cudaStream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const int sms = device_info(dev).sm_count;
    Plan w;
    w.parts = parts_of(a.drafts + a.requests + (a.draft ? a.drafts : 0), a.cols, 4 * sms);
    w.part = ((a.cols + w.parts - 1) / w.parts + 7) & ~int64_t(7);
    w.races = parts_of(a.requests, a.cols, 3 * sms);
    w.share = ((a.cols + w.races - 1) / w.races + 7) & ~int64_t(7);
    uint8_t* p = static_cast<uint8_t*>(a.workspace);
    w.stats = reinterpret_cast<float2*>(p);
    p += round16(sizeof(float2) * kMaxParts * static_cast<size_t>(2 * a.drafts + a.requests));
    w.best = reinterpret_cast<unsigned long long*>(p);
    p += round16(sizeof(unsigned long long) * a.requests);
    w.done = reinterpret_cast<unsigned int*>(p);
    const double c = static_cast<double>(a.scale) * 1.4426950408889634074;
    Scale s;
    s.hi = static_cast<float>(c);
    s.lo = static_cast<float>(c - static_cast<double>(s.hi));
    if (a.dtype == kF32) return launch<float>(a, w, s, stream);
    if (a.dtype == kF16) return launch<__half>(a, w, s, stream);
    return launch<__nv_bfloat16>(a, w, s, stream);
}

}  // namespace lik
