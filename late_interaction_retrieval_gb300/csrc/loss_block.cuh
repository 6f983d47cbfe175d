// loss_block.cuh -- the training objectives over rows of middling length: one
// block a row, the row in its registers.
//
// A row's 16-byte granules are dealt out to the threads, up to kBlockN each; the
// few elements before and after them are one a thread.  All loads are issued at
// once, the warps' statistics meet at one barrier, and every thread turns its
// granules into the gradient and stores them.  A teacher's entries are dealt out
// too: probabilities and their sums beside the row's, and after a second barrier
// the entries' columns are written over the stored row.  A row that is left out
// costs its block one load, and the next block takes its place, so that masks
// need no plan.
//
// Other rows' blocks on the SM cover a row's latencies: 64 registers a thread
// leave room for eight rows of 16 KB.  Twice the threads with half the granules
// were slower (16 KB rows 55 us, 50), and so were half as many registers' worth
// of rows (52).  Measured (8192 rows of bf16, a step with the sum, 16 KB a row):
// policy 48 us, where its bytes take 40; distillation from 64 entries 66, where
// the second barrier and the entries' chain of latencies show; of fp32 47.
#pragma once

#include "dtype_load.cuh"
#include "lik_internal.h"
#include "loss_math.cuh"
#include "losses.h"

namespace lik {
namespace loss {

constexpr int kBlockN = 8;  // granules a thread
constexpr int64_t kBlockBytes = 40960;
constexpr int kBlockWarps = kBlockBytes / (32 * kBlockN * 16);

// The teacher's entries of a row in shared memory: column (-1: padding), the
// teacher's logit and then its probability, the student's logit; and the
// duplicate filter's two bit sets.
struct RowEntries {
    int* index;
    float *p, *z;
    uint32_t *seen, *twice;
    int words;
    // four times the bits that are enough elsewhere: the block waits for what is compared in vain
    static int filter(int k) { return 4 * filter_words(k); }
    static size_t bytes(int k) { return 12u * k + 8u * filter(k); }
    __device__ RowEntries(void* base, int k, int filter_words) : words(filter_words) {
        index = static_cast<int*>(base);
        p = reinterpret_cast<float*>(index + k);
        z = p + k;
        seen = reinterpret_cast<uint32_t*>(z + k);
        twice = seen + words;
    }
    // One warp, entry k of column i a lane: what its column is to get, the sum over
    // all entries of the column in a fixed order; -1 if an earlier entry has it.
    __device__ __forceinline__ float share(int k, int i, int n, int lane) const {
        float mine = i >= 0 ? p[k] : -1.0f;
        bool maybe = false;
        if (i >= 0) {
            const uint32_t h = filter_hash(i, words);
            maybe = twice[h >> 5] >> (h & 31) & 1;
        }
        for (uint32_t todo = __ballot_sync(0xffffffffu, maybe); todo; todo &= todo - 1) {
            const int src = __ffs(todo) - 1, column = __shfl_sync(0xffffffffu, i, src), at = __shfl_sync(0xffffffffu, k, src);
            float sum = 0.0f;
            bool before = false;
            for (int j = lane; j < n; j += 32)
                if (index[j] == column) sum += p[j], before = before || j < at;
            sum = warp_sum(sum);
            before = __any_sync(0xffffffffu, before);
            if (lane == src) mine = before ? -1.0f : sum;
        }
        return mine;
    }
};

template <typename T, int kHead, int kForm>
__global__ void __launch_bounds__(kBlockWarps * 32, 3) loss_block_kernel(const LossRows L, int filter) {
    constexpr int kN = kBlockN;
    constexpr int kV = 16 / sizeof(T);
    constexpr bool kDistill = kHead == kHeadDistill, kGrad = kForm != kFwd, kStat = kForm != kBwd;
    extern __shared__ __align__(16) unsigned char entries[];
    __shared__ Stat parts[kBlockWarps], teacher_parts[kBlockWarps];
    __shared__ float2 loss_parts[kBlockWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x, warps = nt >> 5;
    const int cols = static_cast<int>(L.cols);
    const float c = L.c;
    const int64_t r = blockIdx.x;
    grid_launch_dependents();
    grid_wait();
    const T* z = static_cast<const T*>(L.logits) + r * L.stride;
    T* out = kGrad ? static_cast<T*>(L.grad) + r * L.grad_stride : nullptr;
    const Peek now = peek<kHead, kStat>(L, r);
    const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(T));
    const int head = skew ? kV - skew : 0;  // cols is larger
    const int n = (cols - head) / kV, tail_at = head + n * kV;
    const int loose = tid < head ? tid : tid >= 16 && tid - 16 < cols - tail_at ? tail_at + tid - 16 : -1;
    const bool aligned = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
    const auto store = [&](int g, const uint4& u) {
        T* to = out + head + g * kV;
        if (aligned) *reinterpret_cast<uint4*>(to) = u;
        else store_elements<T>(to, &u);
    };
    const auto zeros = [&] {
        if (kGrad) {
            for (int g = tid; g < n; g += nt) store(g, make_uint4(0, 0, 0, 0));
            if (loose >= 0) out[loose] = from_f32<T>(0.0f);
        }
    };
    if (!kStat && L.sum_out && r == 0 && warp == 0) {  // the loss that this gradient belongs to
        const Sum2 sum = weighted_sum(L.sum_value, L.sum_weight, L.sum_n, lane, 32);
        if (lane == 0) *L.sum_out = static_cast<float>(mean_of(sum.value(), L.sum_weight, L.sum_n));
    }
    // this thread's first entry of the teacher's, before it is known whether the row is read
    int own_i = -1;
    float own_t = -INFINITY;
    if (kDistill && tid < L.k) {
        own_i = L.t_index[r * L.k + tid];
        own_t = teacher_logit(L, r * L.k + tid);
    }
    if (!is_read<kHead, kStat>(L, now)) {
        if (tid == 0 && kStat) {
            if (kHead != kHeadToken) L.row_loss[r] = 0.0f;
            if (kHead == kHeadPolicy) L.row_logp[r] = 0.0f;
            if (L.state) L.state[r] = make_float4(0.f, 0.f, 0.f, 0.f);
        }
        zeros();
        return;
    }
    const RowEntries e(entries, L.k, filter);
    float zy = 0.0f, old_logp = 0.0f, adv = 0.0f, ref = 0.0f, up = 1.0f, lse = 0.0f;
    uint4 u[kN];
#pragma unroll
    for (int h = 0; h < kN; ++h)
        u[h] = tid + h * nt < n ? *reinterpret_cast<const uint4*>(z + head + (tid + h * nt) * kV) : Granule<T>::nothing();
    const float loose_z = loose >= 0 ? load_f32(z + loose) : -INFINITY;
    if (!kStat && L.grad_loss) up = *L.grad_loss;
    if (!kDistill) zy = load_f32(z + now.y);
    if (kHead == kHeadPolicy && kStat) {
        old_logp = L.old_logp[r];
        adv = L.advantage[r];
        if (L.ref_logp) ref = L.ref_logp[r];
    }
    float own_z = 0.0f;
    if (kDistill) {  // entries are dealt out to the threads; a thread comes back to its own
        if (L.t_lse) lse = L.t_lse[r];
        if (own_i >= cols || own_t == -INFINITY) own_i = -1;
        if (own_i >= 0) own_z = load_f32(z + own_i);
        if (kGrad)
            for (int i = tid; i < 2 * e.words; i += nt) e.seen[i] = 0;
        Stat t = {-INFINITY, 0.0f};
        if (warp * 32 < L.k) {
            float top = -INFINITY;
            for (int k = tid; k < L.k; k += nt) {
                if (k != tid) {
                    own_i = L.t_index[r * L.k + k];
                    own_t = teacher_logit(L, r * L.k + k);
                    if (own_i >= cols || own_t == -INFINITY) own_i = -1;
                    e.z[k] = own_i >= 0 ? load_f32(z + own_i) : 0.0f;
                }
                if (own_i < 0) own_i = -1, own_t = -INFINITY;
                e.index[k] = own_i;
                e.p[k] = own_t;
                top = fmaxf(top, own_t);
            }
            t.m = L.t_lse ? 0.0f : warp_max(top);
            for (int k = tid; k < L.k; k += nt)
                t.s += L.t_lse ? ex2((e.p[k] * L.scale - lse) * kLog2e) : ex2((e.p[k] - offset_of(t.m)) * c);
            t.s = warp_sum(t.s);
        }
        if (lane == 0) teacher_parts[warp] = t;
    }
    if (kStat) {
        Running v;
        v.add(loose_z, c);
        v.add_granules<T, kN>(u, c);
        const Stat total = warp_merge(v.stat(), c);
        if (lane == 0) parts[warp] = total;
    }
    if (kDistill && tid < L.k) e.z[tid] = own_z;
    // The row may be written (in place of the logits) from here on.
    __syncthreads();
    float m = now.st.x, inv = now.st.y, s = 0.0f;
    bool live = true;
    if (kStat) {
        Stat total = {-INFINITY, 0.0f};
        if (lane < warps) total = parts[lane];
        total = warp_merge(total, c);
        s = total.s;
        live = s != 0.0f;
        m = offset_of(total.m);
        inv = live ? 1.0f / s : 0.0f;
    }
    float a = 0.0f, coef = 0.0f, at_target = 0.0f, log_ratio = 0.0f;
    if (kDistill) {
        Stat t = {-INFINITY, 0.0f};
        if (lane < warps) t = teacher_parts[lane];
        t = warp_merge(t, c);
        const float base = L.t_lse ? 0.0f : offset_of(t.m), shift = L.t_lse ? lse : logf(t.s);
        // without a normaliser given, probabilities add up to 1 (to NaN, if a logit of theirs is one)
        float mass = L.t_lse ? t.s : t.s != 0.0f ? t.s / t.s : 0.0f;
        if (!kStat) mass = now.st.w;
        live = live && mass != 0.0f;
        coef = kStat ? now.w * L.scale : now.st.z * up * L.scale;
        a = coef * mass * inv;
        float gap = 0.0f, sum = 0.0f;
        if (live && warp * 32 < L.k) {
            for (int k = tid; k < L.k; k += nt) {
                float p = 0.0f;
                if (e.p[k] != -INFINITY) {
                    const float y = (e.p[k] - base) * L.scale;
                    p = ex2((y - shift) * kLog2e);
                    if (kStat && p != 0.0f) gap += p * (y - (e.z[k] - m) * L.scale);
                    if (kGrad) {
                        const uint32_t h = filter_hash(e.index[k], e.words), bit = 1u << (h & 31);
                        if (atomicOr(&e.seen[h >> 5], bit) & bit) atomicOr(&e.twice[h >> 5], bit);
                    }
                }
                e.p[k] = p;
                sum += p;
            }
            if (kStat) gap = warp_sum(gap), sum = warp_sum(sum);
        }
        if (kStat) {
            if (lane == 0) loss_parts[warp] = make_float2(gap, sum);
            if (tid == 0 && L.state) L.state[r] = live ? make_float4(m, inv, now.w, mass) : make_float4(0.f, 0.f, 0.f, 0.f);
            log_ratio = shift - logf(s);
        }
    } else {
        float hot;
        if (kStat) {
            const float lp = live ? (zy - m) * L.scale - logf(s) : 0.0f;
            float2 h = make_float2(0.0f, 0.0f);
            if (kHead == kHeadPolicy && live) {
                h = policy_head(L, lp, old_logp, adv, ref);
                h.y *= now.w;
            }
            if (tid == 0) {
                if (kHead == kHeadPolicy) {
                    L.row_loss[r] = h.x;
                    L.row_logp[r] = lp;
                }
                if (L.state) L.state[r] = live ? make_float4(m, inv, lp, h.y) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
            hot = h.y * L.scale;
        } else {
            hot = now.st.w * up * L.scale;
        }
        a = -hot * inv;
        at_target = target_gradient(zy, m, a, hot, c);
    }
    if (kGrad && live) {
#pragma unroll
        for (int h = 0; h < kN; ++h) {
            const int g = tid + h * nt;
            if (g >= n) break;
            store(g, gradient<T>(u[h], m, a, c));
            if (!kDistill && static_cast<unsigned>(now.y - head - g * kV) < kV) out[now.y] = from_f32<T>(at_target);
        }
        if (loose >= 0) out[loose] = from_f32<T>(!kDistill && loose == now.y ? at_target : a * ex2((loose_z - m) * c));
    } else {
        zeros();
    }
    if (!kDistill) return;
    __syncthreads();
    if (kGrad && live) {  // over what was just stored, at the teacher's columns
        for (int k0 = warp * 32; k0 < L.k; k0 += nt) {
            const int k = k0 + lane, i = k < L.k ? e.index[k] : -1;
            const float p = e.share(k, i, L.k, lane);
            if (!(p < 0.0f)) out[i] = from_f32<T>(a * ex2((e.z[k] - m) * c) - coef * p);
        }
    }
    if (kStat && warp == 0) {
        float2 v = make_float2(0.0f, 0.0f);
        if (lane < warps) v = loss_parts[lane];
        const float gap = warp_sum(v.x), sum = warp_sum(v.y);
        if (lane == 0) L.row_loss[r] = live ? gap - sum * log_ratio : 0.0f;
    }
}

template <typename T, int kHead, int kForm>
cudaError_t launch_block(const LossRows& L, cudaStream_t stream) {
    const int filter = kHead == kHeadDistill ? RowEntries::filter(L.k) : 0;
    const int64_t granules = L.cols / (16 / static_cast<int64_t>(sizeof(T))), each = 32 * kBlockN;
    auto kernel = loss_block_kernel<T, kHead, kForm>;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(static_cast<unsigned>(L.rows));
    lc.blockDim = dim3(static_cast<unsigned>((granules + each - 1) / each * 32));
    lc.dynamicSmemBytes = kHead == kHeadDistill ? RowEntries::bytes(L.k) : 0;
    lc.stream = stream;
    lc.attrs = &attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kernel, L, filter);
}

}  // namespace loss
}  // namespace lik
