// loss_math.cuh -- arithmetic of the training objectives: row softmax
// statistics, the loss heads, and the teacher's entries.
//
// A row's statistics are its max m and S = sum exp(s (z - m)), held in fp32;
// exponentials are taken to base 2, e = 2^(c (z - m)) with c = s log2(e)
// rounded to fp32.  The same c is used everywhere, so that its rounding (6e-8)
// is one of the scale s and of nothing else.  m is subtracted before c is
// applied, so rows of the type's lowest value, whose product with c would
// overflow, need no special case.
#pragma once

#include "dtype_load.cuh"
#include "lik_internal.h"
#include "losses.h"

namespace lik {
namespace loss {

constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Programmatic dependent launch: from here on the stream's next launch may
// start, if it was made to overlap; and the previous launch's writes are there.
__device__ __forceinline__ void grid_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void grid_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// A sum in two fp32 parts: what an addition rounds off is kept.  (As exact as
// fp64 here, whose additions take an SM 16 cycles a warp.)
struct Sum2 {
    float hi = 0.0f, lo = 0.0f;
    __device__ __forceinline__ void add(float x) {
        const float t = hi + x, y = t - hi;
        lo += (hi - (t - y)) + (x - y);
        hi = t;
    }
    __device__ __forceinline__ void add(Sum2 b) {
        add(b.hi);
        lo += b.lo;
    }
    // over the warp, in a fixed order
    __device__ __forceinline__ void reduce() {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            Sum2 b;
            b.hi = __shfl_xor_sync(0xffffffffu, hi, o);
            b.lo = __shfl_xor_sync(0xffffffffu, lo, o);
            add(b);
        }
    }
    // A sum that is not finite has rubbish in lo.
    __device__ __forceinline__ double value() const { return isfinite(hi) ? static_cast<double>(hi) + lo : hi; }
};

// This thread's share (of `threads`, whole warps) of sum weight * value, then
// its warp's, in a fixed order.  weight nullptr: 1 each; a value of 0 adds
// nothing whatever its weight.
__device__ __forceinline__ Sum2 weighted_sum(const float* value, const float* weight, int64_t n, int thread, int threads) {
    Sum2 s;
    int64_t i = thread;
    for (; i + 7 * threads < n; i += 8 * threads) {  // eight loads in flight
        float v[8], w[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            v[k] = value[i + k * threads];
            w[k] = weight ? weight[i + k * threads] : 1.0f;
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (v[k] != 0.0f) s.add(v[k] * w[k]);
    }
    for (; i < n; i += threads) {
        const float v = value[i];
        if (v != 0.0f) s.add(weight ? weight[i] * v : v);
    }
    s.reduce();
    return s;
}
// What a sum without weights is divided by.
__device__ __forceinline__ double mean_of(double sum, const float* weight, int64_t n) {
    return weight || n == 0 ? sum : sum / static_cast<double>(n);
}

// ------------------------------------------------ pairs of fp32 (sm_100) --

struct F2 {
    unsigned long long v;
};
__device__ __forceinline__ F2 f2(float x, float y) {
    F2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(x), "f"(y));
    return r;
}
__device__ __forceinline__ float2 split(F2 a) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(a.v));
    return r;
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
    F2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    F2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
    return r;
}
// ---------------------------------------- 16 bytes of a row as fp32 pairs --

template <typename T>
struct Granule;
// (nothing: -inf throughout.)
template <>
struct Granule<float> {
    static constexpr int kPairs = 2;
    static __device__ __forceinline__ uint4 nothing() { return make_uint4(0xff800000u, 0xff800000u, 0xff800000u, 0xff800000u); }
    static __device__ __forceinline__ float top(const uint4& u) {
        return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
    }
    static __device__ __forceinline__ void widen(const uint4& u, float2 (&x)[2]) {
        x[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
        x[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
    }
    static __device__ __forceinline__ uint4 narrow(const float2 (&x)[2]) {
        return make_uint4(__float_as_uint(x[0].x), __float_as_uint(x[0].y), __float_as_uint(x[1].x), __float_as_uint(x[1].y));
    }
};
template <>
struct Granule<__nv_bfloat16> {
    static constexpr int kPairs = 4;
    static __device__ __forceinline__ uint4 nothing() { return make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }
    static __device__ __forceinline__ __nv_bfloat162 pair(uint32_t w) { return *reinterpret_cast<__nv_bfloat162*>(&w); }
    static __device__ __forceinline__ float top(const uint4& u) {
        const __nv_bfloat162 t = __hmax2(__hmax2(pair(u.x), pair(u.y)), __hmax2(pair(u.z), pair(u.w)));
        return fmaxf(__low2float(t), __high2float(t));
    }
    static __device__ __forceinline__ float2 wide(uint32_t w) {
        return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    }
    static __device__ __forceinline__ void widen(const uint4& u, float2 (&x)[4]) {
        x[0] = wide(u.x), x[1] = wide(u.y), x[2] = wide(u.z), x[3] = wide(u.w);
    }
    static __device__ __forceinline__ uint32_t word(float2 x) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x.x, x.y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ uint4 narrow(const float2 (&x)[4]) {
        return make_uint4(word(x[0]), word(x[1]), word(x[2]), word(x[3]));
    }
};
template <>
struct Granule<__half> {
    static constexpr int kPairs = 4;
    static __device__ __forceinline__ uint4 nothing() { return make_uint4(0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u, 0xfc00fc00u); }
    static __device__ __forceinline__ __half2 pair(uint32_t w) { return *reinterpret_cast<__half2*>(&w); }
    static __device__ __forceinline__ float top(const uint4& u) {
        const __half2 t = __hmax2(__hmax2(pair(u.x), pair(u.y)), __hmax2(pair(u.z), pair(u.w)));
        return fmaxf(__low2float(t), __high2float(t));
    }
    static __device__ __forceinline__ void widen(const uint4& u, float2 (&x)[4]) {
        x[0] = __half22float2(pair(u.x)), x[1] = __half22float2(pair(u.y));
        x[2] = __half22float2(pair(u.z)), x[3] = __half22float2(pair(u.w));
    }
    static __device__ __forceinline__ uint32_t word(float2 x) {
        const __half2 h = __floats2half2_rn(x.x, x.y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
    static __device__ __forceinline__ uint4 narrow(const float2 (&x)[4]) {
        return make_uint4(word(x[0]), word(x[1]), word(x[2]), word(x[3]));
    }
};

// ------------------------------------------------------ row statistics --

// Max and sum of exponentials of a set of logits; none, or -inf alone: (-inf, 0).
struct Stat {
    float m, s;
};

// What is subtracted: 0 in place of -inf, so that logits of -inf give e = 0.
__device__ __forceinline__ float offset_of(float m) { return m == -INFINITY ? 0.0f : m; }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
// One reduction instruction on the bits, ordered as signed integers.  No NaN.
__device__ __forceinline__ float warp_max(float v) {
    int k = __float_as_int(v);
    k ^= (k >> 31) & 0x7fffffff;
    k = __reduce_max_sync(0xffffffffu, k);
    return __int_as_float(k ^ ((k >> 31) & 0x7fffffff));
}

// The statistics of all lanes' sets together.
__device__ __forceinline__ Stat warp_merge(Stat v, float c) {
    const float m = warp_max(v.m);
    return {m, warp_sum(v.s * ex2((v.m - offset_of(m)) * c))};
}

// A thread's running statistics.  A NaN logit leaves the max alone and makes
// the sum NaN.
struct Running {
    float m = -INFINITY;
    F2 s0 = {0}, s1 = {0};

    __device__ __forceinline__ void raise(float top, float c) {
        if (top > m) {
            const float f = ex2((m - top) * c);
            s0 = s0 * f2(f, f);
            s1 = s1 * f2(f, f);
            m = top;
        }
    }
    __device__ __forceinline__ void add(float z, float c) {
        raise(z, c);
        const float x = z - offset_of(m);
        s0 = s0 + f2(ex2(x * c), 0.0f);
    }
    template <typename T, int N>
    __device__ __forceinline__ void add_granules(const uint4 (&u)[N], float c) {
        constexpr int kP = Granule<T>::kPairs;
        float top = Granule<T>::top(u[0]);
#pragma unroll
        for (int i = 1; i < N; ++i) top = fmaxf(top, Granule<T>::top(u[i]));
        raise(top, c);
        const float o = -offset_of(m);
        const F2 off = f2(o, o), cc = f2(c, c);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            float2 x[kP];
            Granule<T>::widen(u[i], x);
#pragma unroll
            for (int j = 0; j < kP; ++j) {
                const float2 y = split((f2(x[j].x, x[j].y) + off) * cc);
                const F2 e = f2(ex2(y.x), ex2(y.y));
                if (j & 1) s1 = s1 + e;
                else s0 = s0 + e;
            }
        }
    }
    __device__ __forceinline__ Stat stat() const {
        const float2 s = split(s0 + s1);
        return {m, s.x + s.y};
    }
};

// ----------------------------------------------------------- gradients --

// a * exp(s (z - m)) of a granule's logits, rounded once.
template <typename T>
__device__ __forceinline__ uint4 gradient(const uint4& u, float m, float a, float c) {
    constexpr int kP = Granule<T>::kPairs;
    float2 x[kP];
    Granule<T>::widen(u, x);
    const F2 off = f2(-m, -m), cc = f2(c, c), aa = f2(a, a);
#pragma unroll
    for (int j = 0; j < kP; ++j) {
        const float2 y = split((f2(x[j].x, x[j].y) + off) * cc);
        x[j] = split(f2(ex2(y.x), ex2(y.y)) * aa);
    }
    return Granule<T>::narrow(x);
}

// The same at a row's target, with the target's own part.
__device__ __forceinline__ float target_gradient(float z, float m, float a, float hot, float c) {
    return fmaf(a, ex2((z - m) * c), hot);
}

// For gradient rows that lie otherwise modulo 16 than their logits.
template <typename T>
__device__ __forceinline__ void store_elements(T* to, const uint4* from) {
    const T* e = reinterpret_cast<const T*>(from);
#pragma unroll
    for (int j = 0; j < static_cast<int>(16 / sizeof(T)); ++j) to[j] = e[j];
}

// ---------------------------------------------------------- row inputs --

// What decides whether a row is read, loaded a row ahead; and its coefficients.
struct Peek {
    int y = -1;
    float w = 1.0f;
    float4 st = {0.0f, 1.0f, 1.0f, 1.0f};
};

template <int kHead, bool kStat>
__device__ __forceinline__ Peek peek(const LossRows& L, int64_t r) {
    Peek p;
    if (r >= L.rows) return p;
    if (kHead != kHeadDistill) p.y = L.target[r];
    if (kStat) p.w = L.weight ? L.weight[r] : L.even_weight;
    else p.st = L.state[r];
    return p;
}

// A row that is left out, or whose gradient has coefficient 0, is not read.
template <int kHead, bool kStat>
__device__ __forceinline__ bool is_read(const LossRows& L, const Peek& p) {
    if (kHead != kHeadDistill && !(p.y >= 0 && p.y < L.cols)) return false;
    if (kStat) return p.w != 0.0f;
    return p.st.y != 0.0f && (kHead == kHeadDistill ? p.st.z : p.st.w) != 0.0f;
}

// The policy loss of a token, and d loss / d log-probability.
__device__ __forceinline__ float2 policy_head(const LossRows& L, float lp, float old_logp, float adv, float ref) {
    const float ratio = expf(lp - old_logp);
    // an advantage of 0 gives no term at a ratio past fp32's range either
    const float inner = adv == 0.0f && ratio == INFINITY ? 0.0f : ratio * adv;
    const float outer = fminf(fmaxf(ratio, 1.0f - L.clip_low), 1.0f + L.clip_high) * adv;
    // the smaller of the two, NaN if either is (fminf would drop it)
    float loss = inner <= outer ? -inner : inner > outer ? -outer : NAN;
    float d = inner <= outer ? -inner : inner > outer ? 0.0f : NAN;
    if (L.ref_logp) {
        const float x = ref - lp, em1 = expm1f(x);  // exp(x) - 1 without cancellation near x = 0
        loss += L.kl_coef * (x == INFINITY ? x : em1 - x);  // of a masked target: not inf - inf
        d -= L.kl_coef * em1;
    }
    return make_float2(loss, d);
}

// --------------------------------------------------- the teacher's entries --

__device__ __forceinline__ float teacher_logit(const LossRows& L, int64_t i) {
    if (L.t_dtype == kF32) return static_cast<const float*>(L.t_logits)[i];
    if (L.t_dtype == kF16) return to_f32(static_cast<const __half*>(L.t_logits)[i]);
    return to_f32(static_cast<const __nv_bfloat16*>(L.t_logits)[i]);
}

}  // namespace loss
}  // namespace lik
