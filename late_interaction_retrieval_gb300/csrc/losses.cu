// losses.cu -- training objectives over rows of logits: what joins the rows
// (pairs of sequences, the loss sum) and the choice of the row kernel.
//
// Every loss here depends on a row only through the log-softmax of its scaled
// logits at a few columns, so with e_c = exp(s (z_c - m)), m the row's max and
// S = sum e_c, the gradient of any of them is
//     g_c = a * e_c + (a sparse part at the target, or at the teacher's columns)
// with one coefficient a per row.
#include "lik_internal.h"
#include "loss_math.cuh"
#include "losses.h"

namespace lik {

cudaError_t launch_loss_f32(LossHead head, LossForm form, const LossRows& L, bool* summed, cudaStream_t stream);
cudaError_t launch_loss_f16(LossHead head, LossForm form, const LossRows& L, bool* summed, cudaStream_t stream);
cudaError_t launch_loss_bf16(LossHead head, LossForm form, const LossRows& L, bool* summed, cudaStream_t stream);

namespace {

cudaError_t launch_dtype(LossHead head, LossForm form, const LossRows& L, bool* summed, cudaStream_t stream) {
    if (L.dtype == kF32) return launch_loss_f32(head, form, L, summed, stream);
    if (L.dtype == kF16) return launch_loss_f16(head, form, L, summed, stream);
    return launch_loss_bf16(head, form, L, summed, stream);
}

__device__ __forceinline__ int64_t clamp_row(int v, int64_t rows) { return v < 0 ? 0 : v > rows ? rows : v; }

constexpr int kPairThreads = 512;
constexpr int kPairWarps = kPairThreads / 64;  // of one sequence

// One block per pair, half of it per sequence: both sequence sums (exact to
// fp32: thousands of log-probabilities enter a small difference), the pair's
// loss, and every row's d loss / d log-probability into its state.  Latency
// bounds it: what does not depend on the sums is loaded before them, and fp64 (a
// division of it above all) is one warp's work: by every thread it held 24 pairs
// of means up by 10 us (1501 x 20011 fp32, a step: 59 us, now 49).
__global__ void __launch_bounds__(kPairThreads) loss_pairs_kernel(const LossPairs P) {
    __shared__ loss::Sum2 part[2][kPairWarps];
    __shared__ int count[2][kPairWarps];
    __shared__ float slope[2];  // d loss / d log-probability of a row
    loss::grid_launch_dependents();
    loss::grid_wait();
    const int64_t p = blockIdx.x;
    const int h = threadIdx.x >= kPairThreads / 2, t = threadIdx.x % (kPairThreads / 2);
    const int64_t seq = p + h * P.pairs;
    // 64 bits: a sequence may end at row 2^31 - 1, and the strides below go past its end
    const int64_t lo = clamp_row(P.offsets[seq], P.rows), hi = clamp_row(P.offsets[seq + 1], P.rows);
    const float w = P.weight ? P.weight[p] : 1.0f / static_cast<float>(P.pairs);
    float ref_chosen = 0.0f, ref_rejected = 0.0f;
    if (P.ref_logp) ref_chosen = P.ref_logp[p], ref_rejected = P.ref_logp[p + P.pairs];
    loss::Sum2 s;
    int n = 0;
    for (int64_t r = lo + t; r < hi; r += kPairThreads / 2) {
        const float4 st = P.state[r];
        if (st.y != 0.0f) {
            s.add(st.z);
            ++n;
        }
    }
    s.reduce();
    n = __reduce_add_sync(0xffffffffu, n);
    if ((threadIdx.x & 31) == 0) {
        part[h][t >> 5] = s;
        count[h][t >> 5] = n;
    }
    __syncthreads();
    if (threadIdx.x < 32) {  // fp64 is slow here: one warp, a sequence a lane
        const int q = threadIdx.x & 1;
        loss::Sum2 all = part[q][0];
        int rows = count[q][0];
        for (int i = 1; i < kPairWarps; ++i) {
            all.add(part[q][i]);
            rows += count[q][i];
        }
        double value = all.value();
        float share = 1.0f;
        if (P.average && rows > 0) {
            value /= rows;
            share = 1.0f / static_cast<float>(rows);
        }
        const double other = __shfl_xor_sync(0xffffffffu, value, 1);
        float g = 0.0f, loss = 0.0f;
        if (w != 0.0f) {
            // of the sums before they are rounded to the fp32 that is returned, whose step (2^-8 at 40000) would
            // show in the loss
            const double gap = (q ? other - value : value - other) - (static_cast<double>(ref_chosen) - ref_rejected);
            const float x = static_cast<float>(P.beta * gap - P.margin);
            const float tail = log1pf(expf(-fabsf(x)));
            // a side without a share has no part in it, though its own loss be infinite (x is where a
            // sequence counts a masked column)
            if (P.smoothing < 1.0f) loss += (1.0f - P.smoothing) * (fmaxf(-x, 0.0f) + tail);
            if (P.smoothing > 0.0f) loss += P.smoothing * (fmaxf(x, 0.0f) + tail);
            if (isnan(x)) loss = x;  // fmaxf drops a NaN
            // sigma(x) - (1 - smoothing), each part without cancellation
            const float pos = 1.0f / (1.0f + expf(-x)), neg = 1.0f / (1.0f + expf(x));
            g = w * P.beta * (P.smoothing * pos - (1.0f - P.smoothing) * neg);
        }
        if (threadIdx.x < 2) {
            P.seq_logp[p + q * P.pairs] = static_cast<float>(value);
            if (q == 0) P.pair_loss[p] = loss;
            slope[q] = (q ? -g : g) * share;
        }
    }
    __syncthreads();
    const float v = slope[h];
    for (int64_t r = lo + t; r < hi; r += kPairThreads / 2)
        if (P.state[r].y != 0.0f) P.state[r].w = v;
}

constexpr int kSumThreads = 1024;

__global__ void __launch_bounds__(kSumThreads)
loss_sum_kernel(const float* value, const float* weight, int64_t n, float* loss) {
    __shared__ loss::Sum2 part[kSumThreads / 32];
    loss::grid_launch_dependents();
    loss::grid_wait();
    const loss::Sum2 s = loss::weighted_sum(value, weight, n, threadIdx.x, kSumThreads);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x < 32) {
        loss::Sum2 r = part[threadIdx.x];
        r.reduce();
        if (threadIdx.x == 0) *loss = static_cast<float>(loss::mean_of(r.value(), weight, n));
    }
}

// One launch, which may start while the one before it on the stream ends: every
// kernel here waits for that one's writes before it touches memory.
template <typename... Params, typename... Args>
cudaError_t launch(void (*kernel)(Params...), unsigned blocks, int threads, cudaStream_t stream, Args... args) {
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(blocks);
    lc.blockDim = dim3(threads);
    lc.stream = stream;
    lc.attrs = &attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kernel, args...);
}

}  // namespace

cudaError_t launch_loss_rows(LossHead head, const LossRows& L, bool* summed, cudaStream_t stream) {
    if (summed) *summed = false;
    return launch_dtype(head, L.grad ? kStep : kFwd, L, summed, stream);
}

cudaError_t launch_loss_grad(LossHead head, const LossRows& L, cudaStream_t stream) {
    return launch_dtype(head, kBwd, L, nullptr, stream);
}

cudaError_t launch_loss_pairs(const LossPairs& P, cudaStream_t stream) {
    return launch(loss_pairs_kernel, static_cast<unsigned>(P.pairs), kPairThreads, stream, P);
}

cudaError_t launch_loss_sum(const float* value, const float* weight, int64_t n, float* loss, cudaStream_t stream) {
    return launch(loss_sum_kernel, 1, kSumThreads, stream, value, weight, n, loss);
}

}  // namespace lik
