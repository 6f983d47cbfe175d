// loss_rows.cuh -- the row kernel of the training objectives: one block a row,
// softmax statistics, loss head and gradient.
//
// A row's 16-byte granules are dealt out to the threads in batches of kN each;
// the few elements before the first and after the last are one a thread.  A
// batch's loads go out at once and stay in registers while they are summed.  The
// warps' statistics meet at one barrier, after which every thread knows the
// row's coefficients.  A step then turns the batch it still has in registers
// into the gradient and goes back over the others, which come from L2: the rows
// at work are kept few enough, and the gradient is stored past them.  A gradient
// from saved statistics goes over the row once.
//
// A teacher's entries are dealt out over the threads too: their softmax runs
// beside the row's, and after a second barrier the entries' columns are written
// over the stored row.  A row that is left out costs its block a load or two and, with
// a gradient, the row of zeros; the next block takes its place, so that masks need
// no plan.
//
// Memory bounds it; the other rows of an SM cover a row's latencies, which is why
// blocks are as small as the rules at the launch allow.  Measured (bf16, inputs
// beyond L2, a step with the sum; in brackets the time its bytes take at the rate
// of a copy): policy 8192 rows of 16 KB 46 us (40), of 64 KB 159 (155);
// distillation from 64 entries, 4096 rows of 256 KB 353 (309); forward 2048 rows
// of 256 KB 82 (77).  Without the hints on second loads and gradient stores the
// distillation takes 392, 64 KB rows 169.  Rows held in shared memory by clusters
// of CTAs, loaded and stored by bulk copies, took 373 and 181.
#pragma once

#include <algorithm>

#include "dtype_load.cuh"
#include "lik_internal.h"
#include "loss_math.cuh"
#include "losses.h"

namespace lik {
namespace loss {

constexpr int kRowN = 8;       // granules of a thread's batch
constexpr int kRowWarps = 32;  // of a block, at most; 64 registers a thread

// The teacher's entries of a row in shared memory: column (-1: padding), the
// teacher's logit and then its probability, the student's logit.  Duplicate
// columns are found by two bit sets over a hash of the column, so that only the
// few entries that may have a double are compared with others: 64 bits an entry
// at least, one entry in 64 is compared in vain.
struct RowEntries {
    int* index;
    float *p, *z;
    uint32_t *seen, *twice;
    int words;
    static int filter(int k) {
        int n = 128;
        while (n < 2 * k) n *= 2;
        return n;
    }
    static size_t bytes(int k) { return 12u * k + 8u * filter(k); }
    __device__ RowEntries(void* base, int k, int filter_words) : words(filter_words) {
        index = static_cast<int*>(base);
        p = reinterpret_cast<float*>(index + k);
        z = p + k;
        seen = reinterpret_cast<uint32_t*>(z + k);
        twice = seen + words;
    }
    __device__ __forceinline__ uint32_t hash(int column) const {
        return (static_cast<uint32_t>(column) * 2654435761u) >> __clz(words * 32 - 1);  // log2(32 words) bits
    }
    // One warp, entry k of column i a lane: what its column is to get, the sum over
    // all entries of the column in a fixed order; -1 if an earlier entry has it.
    __device__ __forceinline__ float share(int k, int i, int n, int lane) const {
        float mine = i >= 0 ? p[k] : -1.0f;
        bool maybe = false;
        if (i >= 0) {
            const uint32_t h = hash(i);
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
__global__ void __launch_bounds__(kRowWarps * 32, 1) loss_row_kernel(const LossRows L, int filter) {
    constexpr int kN = kRowN;
    constexpr int kV = 16 / sizeof(T);
    constexpr bool kDistill = kHead == kHeadDistill, kGrad = kForm != kFwd, kStat = kForm != kBwd;
    extern __shared__ __align__(16) unsigned char entries[];
    __shared__ Stat parts[kRowWarps], teacher_parts[kRowWarps];
    __shared__ float2 loss_parts[kRowWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nt = blockDim.x, warps = nt >> 5;
    const int cols = static_cast<int>(L.cols);
    const float c = L.c;
    // Backwards the last row first: those a forward read last are the likeliest in L2.
    const int64_t r = kStat ? blockIdx.x : L.rows - 1 - static_cast<int64_t>(blockIdx.x);
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
        T* to = out + head + static_cast<int64_t>(g) * kV;
        if (aligned) __stcs(reinterpret_cast<uint4*>(to), u);
        else store_elements<T>(to, &u);
    };
    const auto zeros = [&] {
        if (kGrad) {
            for (int g = tid; g < n; g += nt) store(g, make_uint4(0, 0, 0, 0));
            if (loose >= 0) out[loose] = from_f32<T>(0.0f);
        }
    };
    if (!kStat && L.sum_out && blockIdx.x == 0 && warp == 0) {  // the loss that this gradient belongs to
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
    const auto load = [&](int g0, bool last) {  // last: not read again
#pragma unroll
        for (int h = 0; h < kN; ++h) {
            const int g = g0 + h * nt;
            const uint4* at = reinterpret_cast<const uint4*>(z + head) + g;
            if (g >= n) u[h] = Granule<T>::nothing();
            else u[h] = last ? __ldcs(at) : *at;
        }
    };
    int batch = 0;
    load(tid, false);
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
                if (e.p[k] != -INFINITY)  // whatever the normaliser, padding has no mass
                    t.s += L.t_lse ? ex2(fmaf(e.p[k], L.scale, -lse) * kLog2e) : ex2((e.p[k] - offset_of(t.m)) * c);
            t.s = warp_sum(t.s);
        }
        if (lane == 0) teacher_parts[warp] = t;
    }
    if (kStat) {
        Running v;
        v.add(loose_z, c);
        v.add_granules<T, kN>(u, c);
        for (int g = kN * nt; g < n; g += kN * nt) {
            load(g + tid, false);
            v.add_granules<T, kN>(u, c);
            batch = g;
        }
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
    float a = 0.0f, coef = 0.0f, at_target = 0.0f, log_s = 0.0f;
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
                    // one rounding: a level that the teacher's logits and lse share cancels here
                    const float log_p = fmaf(e.p[k] - base, L.scale, -shift);
                    p = ex2(log_p * kLog2e);
                    if (kStat && p != 0.0f) gap += p * (log_p - (e.z[k] - m) * L.scale);
                    if (kGrad) {
                        const uint32_t h = e.hash(e.index[k]), bit = 1u << (h & 31);
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
            log_s = logf(s);
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
        while (true) {
#pragma unroll
            for (int h = 0; h < kN; ++h) {
                const int g = batch + tid + h * nt;
                if (g >= n) break;
                store(g, gradient<T>(u[h], m, a, c));
                if (!kDistill && static_cast<unsigned>(now.y - head - g * kV) < kV) out[now.y] = from_f32<T>(at_target);
            }
            batch += kForm == kStep ? -kN * nt : kN * nt;
            if (kForm == kStep ? batch < 0 : batch >= n) break;
            load(batch + tid, true);
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
        if (lane == 0) L.row_loss[r] = live ? gap + sum * log_s : 0.0f;
    }
}

// Warps of a block: 32 fill an SM's registers, in blocks of 8 when nothing speaks
// against it.
//   - Rows that do not fill the SMs take 16 or 32 (152 rows of 256 KB: forward 13
//     us with 16 warps, 23 with 8; a step 20 with 32, 26 and 43).
//   - In a step the rows at work share L2 with the gradient on its way out: blocks
//     of 8 up to half of it (rows of 96 KB 250 us, 257 with 16; of 128 KB 363 and
//     323), of 16 up to three quarters (160 KB 429, 593 with 32; distillation 256 KB
//     353 and 378; fp32 400 KB 249 and 235).
//   - Two batches a thread at least: a block's second loads cover its first sums
//     (forward 16 KB 26 us, 29 with one; 32 KB 44 and 51; distillation step 32 KB 93
//     and 104).  Batches are of equal size.
//   - A warp for 224 of a teacher's entries at least (8192 x 4000 bf16, a step: 256
//     entries 49 us, 62 by one warp; 1000 entries 123 by five, 360 by one; but
//     8192 x 1000 fp32 200 entries 35, 42 by two).  Those are 2.3, 4.2 and 3.1 times
//     what their bytes take: an entry's loads depend on one another, and it ends as
//     a store of its own.
inline int row_warps(int64_t rows, int64_t row_bytes, int entries, bool step, const DeviceInfo& dev) {
    const int64_t at_once = row_bytes * dev.sm_count;  // by blocks of 32
    int most = 8;
    if (rows <= 2 * dev.sm_count || (step && 4 * at_once > dev.l2_bytes / 2)) most = 16;
    if (rows <= dev.sm_count || (step && 2 * at_once > dev.l2_bytes / 4 * 3)) most = kRowWarps;
    const int64_t batch = 32 * kRowN * 16;
    const int64_t batches = row_bytes <= 2 * most * batch ? 2 : (row_bytes + most * batch - 1) / (most * batch);
    const int warps = static_cast<int>((row_bytes + batches * batch - 1) / (batches * batch));
    return std::max(warps, (entries + 223) / 224);
}

template <typename T, int kHead, int kForm>
cudaError_t launch_rows_kernel(const LossRows& L, cudaStream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const int filter = kHead == kHeadDistill ? RowEntries::filter(L.k) : 0;
    const int warps = row_warps(L.rows, L.cols * static_cast<int64_t>(sizeof(T)), kHead == kHeadDistill ? L.k : 0, kForm == kStep,
                                device_info(dev));
    auto kernel = loss_row_kernel<T, kHead, kForm>;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(static_cast<unsigned>(L.rows));
    lc.blockDim = dim3(static_cast<unsigned>(warps * 32));
    lc.dynamicSmemBytes = kHead == kHeadDistill ? RowEntries::bytes(L.k) : 0;
    lc.stream = stream;
    lc.attrs = &attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kernel, L, filter);
}

}  // namespace loss
}  // namespace lik
