// losses.cu -- training objectives over rows of logits: row softmax
// statistics, the loss heads on them, and the gradient.
//
// Every loss here depends on a row only through the log-softmax of its scaled
// logits at a few columns, so with e_c = exp(s (z_c - m)), m the row's max and
// S = sum e_c, the gradient of any of them is
//     g_c = a * e_c + (a sparse part at the target, or at the teacher's columns)
// with one coefficient a per row.
#include "dtype_load.cuh"
#include "lik_internal.h"
#include "losses.h"

namespace lik {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
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

// Max and scaled sum of exponentials of a set of logits; the set of none (or
// of -inf alone) is (-inf, 0).
struct Stat {
    float m, s;
};

// The offset to subtract: 0 in place of -inf, so that -inf logits give e = 0.
__device__ __forceinline__ float offset_of(float m) { return m == -INFINITY ? 0.0f : m; }

__device__ __forceinline__ Stat merge(Stat a, Stat b, float c) {
    const float m = fmaxf(a.m, b.m), o = offset_of(m);
    return {m, a.s * ex2((a.m - o) * c) + b.s * ex2((b.m - o) * c)};
}

__device__ __forceinline__ Stat warp_merge(Stat v, float c) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        v = merge(v, {__shfl_xor_sync(0xffffffffu, v.m, o), __shfl_xor_sync(0xffffffffu, v.s, o)}, c);
    return v;
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, o));
    return v;
}

// Block-wide results, the same in every thread.  `part` is reused: callers
// may call again at once.
__device__ Stat block_merge(Stat v, float c, float2* part) {
    v = warp_merge(v, c);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = make_float2(v.m, v.s);
    __syncthreads();
    Stat r = {part[0].x, part[0].y};
    for (int w = 1; w < kWarps; ++w) r = merge(r, {part[w].x, part[w].y}, c);
    return r;
}
__device__ float2 block_sum2(float x, float y, float2* part) {
    x = warp_sum(x);
    y = warp_sum(y);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = make_float2(x, y);
    __syncthreads();
    float2 r = part[0];
    for (int w = 1; w < kWarps; ++w) {
        r.x += part[w].x;
        r.y += part[w].y;
    }
    return r;
}

// The policy head at one token: its loss and d loss / d log-probability.
__device__ __forceinline__ float2 policy_head(const LossRows& L, int64_t r, float lp) {
    const float adv = L.advantage[r];
    const float ratio = expf(lp - L.old_logp[r]);
    const float inner = ratio * adv;
    const float outer = fminf(fmaxf(ratio, 1.0f - L.clip_low), 1.0f + L.clip_high) * adv;
    // the smaller of the two, NaN if either is (fminf would drop it)
    float loss = inner <= outer ? -inner : inner > outer ? -outer : NAN;
    float d = inner <= outer ? -inner : inner > outer ? 0.0f : NAN;
    if (L.ref_logp) {
        const float x = L.ref_logp[r] - lp, em1 = expm1f(x);  // exp(x) - 1 without cancellation near x = 0
        loss += L.kl_coef * (em1 - x);
        d -= L.kl_coef * em1;
    }
    return make_float2(loss, d);
}

__device__ __forceinline__ float teacher_at(const LossRows& L, int64_t i) {
    if (L.t_dtype == kF32) return static_cast<const float*>(L.t_logits)[i];
    if (L.t_dtype == kF16) return to_f32(static_cast<const __half*>(L.t_logits)[i]);
    return to_f32(static_cast<const __nv_bfloat16*>(L.t_logits)[i]);
}

// One block per row (grid-stride).  kFwd: statistics and loss from the
// logits; otherwise they come from the row state.  kGrad: the gradient.
template <typename T, int kHead, bool kFwd, bool kGrad>
__global__ void __launch_bounds__(kThreads) loss_rows_kernel(const LossRows L) {
    __shared__ float2 part[kWarps];
    __shared__ int t_idx[kHead == kHeadDistill ? kMaxTeacher : 1];
    __shared__ float t_p[kHead == kHeadDistill ? kMaxTeacher : 1];
    __shared__ float t_z[kHead == kHeadDistill ? kMaxTeacher : 1];
    const int tid = threadIdx.x;
    const int cols = static_cast<int>(L.cols);
    const float c = L.scale * kLog2e;
    const float up = !kFwd && L.grad_loss ? *L.grad_loss : 1.0f;
    for (int64_t r = blockIdx.x; r < L.rows; r += gridDim.x) {
        const T* z = static_cast<const T*>(L.logits) + r * L.stride;
        T* g = kGrad ? static_cast<T*>(L.grad) + r * L.grad_stride : nullptr;
        const float w = !kFwd ? 1.0f : L.weight ? L.weight[r] : 1.0f / static_cast<float>(L.rows);
        int y = -1;
        if (kHead != kHeadDistill) y = L.target[r];
        bool live = w != 0.0f && (kHead == kHeadDistill || (y >= 0 && y < cols));
        float4 st = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (!kFwd) {
            st = L.state[r];
            live = live && st.y != 0.0f && (kHead == kHeadDistill ? st.z : st.w) != 0.0f;
        }
        if (live && kHead == kHeadDistill) {  // the teacher's probabilities and the student's logits there
            __syncthreads();
            float mt = -INFINITY;
            for (int k = tid; k < L.k; k += kThreads) {
                const int i = L.t_index[r * L.k + k];
                const bool in = i >= 0 && i < cols;
                const float t = in ? teacher_at(L, r * L.k + k) : -INFINITY;
                t_idx[k] = in ? i : -1;
                t_p[k] = t;
                t_z[k] = in ? load_f32(z + i) : 0.0f;
                mt = fmaxf(mt, t);
            }
            Stat ts = {mt, 0.0f};
            for (int k = tid; k < L.k; k += kThreads) ts.s += ex2((t_p[k] - offset_of(mt)) * c);
            ts = block_merge(ts, c, part);
            // t_p becomes log p (natural), -inf without mass
            const float shift = L.t_lse ? L.t_lse[r] : logf(ts.s);
            const float base = L.t_lse ? 0.0f : offset_of(ts.m);
            for (int k = tid; k < L.k; k += kThreads)
                if (t_p[k] != -INFINITY) t_p[k] = (t_p[k] - base) * L.scale - shift;
        }
        Stat v = {-INFINITY, 0.0f};
        if (kFwd && live) {
            for (int i = tid; i < cols; i += kThreads) {
                const float x = load_f32(z + i);
                if (x > v.m) {
                    v.s *= ex2((v.m - x) * c);
                    v.m = x;
                }
                v.s += ex2((x - offset_of(v.m)) * c);
            }
            v = block_merge(v, c, part);
            live = v.s != 0.0f;
        }
        float m = offset_of(v.m), inv = 1.0f / v.s;
        float coef = 0.0f;  // multiplies e_c; the sparse part below
        if (kHead == kHeadDistill) {
            float mass = 0.0f, loss = 0.0f;
            const float log_s = logf(v.s);
            if (live) {
                for (int k = tid; k < L.k; k += kThreads) {
                    const float lp = t_p[k];
                    const float p = t_idx[k] >= 0 ? ex2(lp * kLog2e) : 0.0f;
                    t_p[k] = p;
                    mass += p;
                    if (kFwd && p != 0.0f) loss += p * (lp - ((t_z[k] - m) * L.scale - log_s));
                }
                const float2 sums = block_sum2(mass, loss, part);
                mass = sums.x;
                loss = sums.y;
            }
            if (kFwd) {
                live = live && mass != 0.0f;
                if (tid == 0) {
                    L.row_loss[r] = live ? loss : 0.0f;
                    if (L.state) L.state[r] = live ? make_float4(m, inv, w, mass) : make_float4(0.f, 0.f, 0.f, 0.f);
                }
                coef = w * L.scale;
            } else {
                m = st.x;
                inv = st.y;
                mass = st.w;
                coef = st.z * L.scale * up;
            }
            if (kGrad) {
                const float a = coef * mass * inv;
                for (int i = tid; i < cols; i += kThreads)
                    g[i] = from_f32<T>(live ? a * ex2((load_f32(z + i) - m) * c) : 0.0f);
                __syncthreads();
                if (live)
                    for (int k = tid; k < L.k; k += kThreads) {
                        const int i = t_idx[k];
                        if (i < 0) continue;
                        float p = 0.0f;
                        bool owner = true;
                        for (int j = 0; j < L.k; ++j) {
                            if (t_idx[j] != i) continue;
                            owner = owner && j >= k;
                            p += t_p[j];
                        }
                        if (owner) g[i] = from_f32<T>(a * ex2((t_z[k] - m) * c) - coef * p);
                    }
                __syncthreads();
            }
        } else {
            float hot = 0.0f;
            if (kFwd) {
                const float lp = live ? (load_f32(z + y) - m) * L.scale - logf(v.s) : 0.0f;
                float d = 0.0f;
                if (kHead == kHeadPolicy) {
                    float2 h = make_float2(0.0f, 0.0f);
                    if (live) h = policy_head(L, r, lp);
                    d = h.y * w;
                    if (tid == 0) {
                        L.row_loss[r] = h.x;
                        L.row_logp[r] = lp;
                    }
                }
                if (tid == 0 && L.state) L.state[r] = live ? make_float4(m, inv, lp, d) : make_float4(0.f, 0.f, 0.f, 0.f);
                hot = d * L.scale;
                if (kGrad) __syncthreads();  // in place: every thread has read the target's logit
            } else {
                m = st.x;
                inv = st.y;
                hot = st.w * L.scale * up;
            }
            if (kGrad) {
                for (int i = tid; i < cols; i += kThreads) {
                    float x = 0.0f;
                    if (live) {
                        x = -hot * (ex2((load_f32(z + i) - m) * c) * inv);
                        if (i == y) x += hot;
                    }
                    g[i] = from_f32<T>(x);
                }
            }
        }
    }
}

template <typename T, bool kFwd, bool kGrad>
cudaError_t launch_head(LossHead head, const LossRows& L, cudaStream_t stream) {
    int dev = 0;
    cudaGetDevice(&dev);
    const int64_t cap = static_cast<int64_t>(device_info(dev).sm_count) * 8;
    const unsigned blocks = static_cast<unsigned>(L.rows < cap ? L.rows : cap);
    if (head == kHeadDistill)
        loss_rows_kernel<T, kHeadDistill, kFwd, kGrad><<<blocks, kThreads, 0, stream>>>(L);
    else if (head == kHeadPolicy)
        loss_rows_kernel<T, kHeadPolicy, kFwd, kGrad><<<blocks, kThreads, 0, stream>>>(L);
    else
        loss_rows_kernel<T, kHeadToken, kFwd, kGrad><<<blocks, kThreads, 0, stream>>>(L);
    return cudaGetLastError();
}

template <bool kFwd, bool kGrad>
cudaError_t launch_dtype(LossHead head, const LossRows& L, cudaStream_t stream) {
    if (L.dtype == kF32) return launch_head<float, kFwd, kGrad>(head, L, stream);
    if (L.dtype == kF16) return launch_head<__half, kFwd, kGrad>(head, L, stream);
    return launch_head<__nv_bfloat16, kFwd, kGrad>(head, L, stream);
}

__device__ __forceinline__ int clamp_row(int v, int64_t rows) {
    return v < 0 ? 0 : static_cast<int64_t>(v) > rows ? static_cast<int>(rows) : v;
}

// Block-wide fp64 sums of two values, in a fixed order.
__device__ double2 block_sum_d(double x, double y, double2* part) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        x += __shfl_xor_sync(0xffffffffu, x, o);
        y += __shfl_xor_sync(0xffffffffu, y, o);
    }
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = make_double2(x, y);
    __syncthreads();
    double2 r = part[0];
    for (int w = 1; w < kWarps; ++w) {
        r.x += part[w].x;
        r.y += part[w].y;
    }
    return r;
}

// One block per pair: both sequence sums (fp64: a sum of thousands of
// log-probabilities enters a difference), the pair's loss, and every row's
// d loss / d log-probability into its state.
__global__ void __launch_bounds__(kThreads) loss_pairs_kernel(const LossPairs P) {
    __shared__ double2 part[kWarps];
    const int64_t p = blockIdx.x;
    double sum[2];
    float share[2];
    int lo[2], hi[2];
    for (int h = 0; h < 2; ++h) {
        const int64_t i = p + h * P.pairs;
        lo[h] = clamp_row(P.offsets[i], P.rows);
        hi[h] = clamp_row(P.offsets[i + 1], P.rows);
        double s = 0.0, n = 0.0;
        for (int r = lo[h] + static_cast<int>(threadIdx.x); r < hi[h]; r += kThreads) {
            const float4 st = P.state[r];
            if (st.y != 0.0f) {
                s += st.z;
                n += 1.0;
            }
        }
        const double2 t = block_sum_d(s, n, part);
        share[h] = P.average && t.y > 0.0 ? static_cast<float>(1.0 / t.y) : 1.0f;
        sum[h] = P.average && t.y > 0.0 ? t.x / t.y : t.x;
        if (threadIdx.x == 0) P.seq_logp[i] = static_cast<float>(sum[h]);
    }
    const float w = P.weight ? P.weight[p] : 1.0f / static_cast<float>(P.pairs);
    float g = 0.0f, loss = 0.0f;
    if (w != 0.0f) {
        double gap = sum[0] - sum[1];
        if (P.ref_logp) gap -= static_cast<double>(P.ref_logp[p]) - static_cast<double>(P.ref_logp[p + P.pairs]);
        const float x = static_cast<float>(P.beta * gap - P.margin);
        const float tail = log1pf(expf(-fabsf(x)));
        loss = (1.0f - P.smoothing) * (fmaxf(-x, 0.0f) + tail) + P.smoothing * (fmaxf(x, 0.0f) + tail);
        // sigma(x) - (1 - smoothing), each part without cancellation
        const float pos = 1.0f / (1.0f + expf(-x)), neg = 1.0f / (1.0f + expf(x));
        g = w * P.beta * (P.smoothing * pos - (1.0f - P.smoothing) * neg);
    }
    if (threadIdx.x == 0) P.pair_loss[p] = loss;
    for (int h = 0; h < 2; ++h) {
        const float v = (h ? -g : g) * share[h];
        for (int r = lo[h] + static_cast<int>(threadIdx.x); r < hi[h]; r += kThreads)
            if (P.state[r].y != 0.0f) P.state[r].w = v;
    }
}

__global__ void __launch_bounds__(kThreads)
loss_sum_kernel(const float* value, const float* weight, int64_t n, float* loss) {
    __shared__ double2 part[kWarps];
    double s = 0.0;
    for (int64_t i = threadIdx.x; i < n; i += kThreads) {
        const float v = value[i];
        if (v != 0.0f) s += weight ? static_cast<double>(weight[i]) * v : v;
    }
    s = block_sum_d(s, 0.0, part).x;
    if (threadIdx.x == 0) *loss = static_cast<float>(weight || n == 0 ? s : s / static_cast<double>(n));
}

}  // namespace

cudaError_t launch_loss_rows(LossHead head, const LossRows& L, cudaStream_t stream) {
    return L.grad ? launch_dtype<true, true>(head, L, stream) : launch_dtype<true, false>(head, L, stream);
}

cudaError_t launch_loss_grad(LossHead head, const LossRows& L, cudaStream_t stream) {
    return launch_dtype<false, true>(head, L, stream);
}

cudaError_t launch_loss_pairs(const LossPairs& P, cudaStream_t stream) {
    loss_pairs_kernel<<<static_cast<unsigned>(P.pairs), kThreads, 0, stream>>>(P);
    return cudaGetLastError();
}

cudaError_t launch_loss_sum(const float* value, const float* weight, int64_t n, float* loss, cudaStream_t stream) {
    loss_sum_kernel<<<1, kThreads, 0, stream>>>(value, weight, n, loss);
    return cudaGetLastError();
}

}  // namespace lik
