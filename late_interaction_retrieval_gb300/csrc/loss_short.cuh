// loss_short.cuh -- the training objectives over short rows (a query's
// candidates, a small vocabulary): one warp a row, the row in its registers.
//
// What bounds it is latency: a row is a few loads that depend on nothing, two
// warp reductions and its stores (256 rows of 17 fp32 scores, 16 teacher entries,
// a step with the sum: 11.6 us, of which the call's host side is all but 6).  Rows
// of up to 32 * kShortN granules of 16 bytes; the few elements before the first
// granule and after the last are one a lane.  A row's teacher is added up by
// column in shared memory, one float a column.
#pragma once

#include "dtype_load.cuh"
#include "lik_internal.h"
#include "loss_math.cuh"
#include "losses.h"

namespace lik {
namespace loss {

// Adds p to dense[i] for the lanes with i >= 0, lanes of one column in lane
// order; one warp, dense in shared memory.
__device__ __forceinline__ void add_in_order(float* dense, int i, float p, int lane) {
    const uint32_t same = __match_any_sync(0xffffffffu, i);
    if (__all_sync(0xffffffffu, same == 1u << lane || i < 0)) {  // no column twice
        if (i >= 0) dense[i] += p;
    } else {
        const int first = __ffs(same) - 1;
        float sum = 0.0f;
        for (int k = 0; k < 32; ++k) {
            const float v = __shfl_sync(0xffffffffu, p, k);
            if (same >> k & 1) sum += v;
        }
        if (i >= 0 && lane == first) dense[i] += sum;
    }
    __syncwarp();
}

constexpr int kShortN = 2;
constexpr int64_t kShortBytes = 32 * kShortN * 16;

template <typename T, int kHead, int kForm>
__global__ void __launch_bounds__(1024) loss_short_kernel(const LossRows L) {
    constexpr int kN = kShortN, kV = 16 / sizeof(T), kP = Granule<T>::kPairs;
    constexpr bool kDistill = kHead == kHeadDistill, kGrad = kForm != kFwd, kStat = kForm != kBwd;
    extern __shared__ float dense_all[];
    __shared__ Sum2 part[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
    const int cols = static_cast<int>(L.cols);
    float* dense = dense_all + warp * cols;  // the teacher's probabilities by column
    const float c = L.c;
    grid_launch_dependents();
    grid_wait();
    const float up = !kStat && L.grad_loss ? *L.grad_loss : 1.0f;
    const int64_t step = static_cast<int64_t>(gridDim.x) * warps;
    int64_t r = static_cast<int64_t>(blockIdx.x) * warps + warp;
    Peek next = peek<kHead, kStat>(L, r);
    for (; r < L.rows; r += step) {
        const Peek now = next;
        next = peek<kHead, kStat>(L, r + step);
        const T* z = static_cast<const T*>(L.logits) + r * L.stride;
        T* out = kGrad ? static_cast<T*>(L.grad) + r * L.grad_stride : nullptr;
        const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(z) & 15) / sizeof(T));
        const int head = min(skew ? kV - skew : 0, cols);
        const int n = (cols - head) / kV, tail_at = head + n * kV;
        const int loose = lane < head ? lane : lane >= 16 && lane - 16 < cols - tail_at ? tail_at + lane - 16 : -1;
        const bool read = is_read<kHead, kStat>(L, now);
        uint4 u[kN];
        float loose_z = -INFINITY, zy = 0.0f, old_logp = 0.0f, adv = 0.0f, ref = 0.0f;
#pragma unroll
        for (int h = 0; h < kN; ++h) u[h] = Granule<T>::nothing();
        if (read) {
#pragma unroll
            for (int h = 0; h < kN; ++h)
                if (lane + 32 * h < n) u[h] = *reinterpret_cast<const uint4*>(z + head + (lane + 32 * h) * kV);
            if (loose >= 0) loose_z = load_f32(z + loose);
            if (!kDistill) zy = load_f32(z + now.y);
            if (kHead == kHeadPolicy && kStat) {
                old_logp = L.old_logp[r];
                adv = L.advantage[r];
                if (L.ref_logp) ref = L.ref_logp[r];
            }
        }
        float m = 0.0f, inv = 0.0f, log_s = 0.0f;
        bool live = read;
        if (kStat && read) {
            Running v;
            v.add(loose_z, c);
            v.add_granules<T, kN>(u, c);
            const Stat total = warp_merge(v.stat(), c);
            live = total.s != 0.0f;
            m = offset_of(total.m);
            inv = live ? 1.0f / total.s : 0.0f;
            log_s = logf(total.s);
        }
        float a = 0.0f, coef = 0.0f, at_target = 0.0f;
        if (kDistill) {
            float mass = 0.0f, gap = 0.0f, loss = 0.0f;
            if (live) {
                // the teacher: its max, its sum, then p and what follows from it
                const int32_t* index = L.t_index + r * L.k;
                float base = 0.0f, shift = 0.0f;
                if (L.t_lse) {
                    shift = L.t_lse[r];
                } else {
                    float top = -INFINITY, s = 0.0f;
                    for (int k = lane; k < L.k; k += 32) {
                        const int i = index[k];
                        if (i >= 0 && i < cols) top = fmaxf(top, teacher_logit(L, r * L.k + k));
                    }
                    base = offset_of(warp_max(top));
                    for (int k = lane; k < L.k; k += 32) {
                        const int i = index[k];
                        if (i >= 0 && i < cols) s += ex2((teacher_logit(L, r * L.k + k) - base) * c);
                    }
                    shift = logf(warp_sum(s));
                }
                if (kGrad) {
                    for (int i = lane; i < cols; i += 32) dense[i] = 0.0f;
                    __syncwarp();
                }
                for (int k0 = 0; k0 < L.k; k0 += 32) {
                    const int k = k0 + lane;
                    int i = k < L.k ? index[k] : -1;
                    float p = 0.0f;
                    if (i >= cols) i = -1;
                    if (i >= 0) {
                        const float t = teacher_logit(L, r * L.k + k);
                        if (t != -INFINITY) {
                            // one rounding: a level that the teacher's logits and lse share cancels here
                            const float log_p = fmaf(t - base, L.scale, -shift);
                            p = ex2(log_p * kLog2e);
                            if (kStat && p != 0.0f) gap += p * (log_p - (load_f32(z + i) - m) * L.scale);
                        }
                        mass += p;
                    }
                    if (kGrad) add_in_order(dense, i < 0 ? -1 : i, p, lane);
                }
                mass = warp_sum(mass);
                if (kStat) {
                    loss = warp_sum(gap) + mass * log_s;
                    live = mass != 0.0f;
                }
            }
            if (kStat) {
                if (lane == 0) {
                    L.row_loss[r] = live ? loss : 0.0f;
                    if (L.state) L.state[r] = live ? make_float4(m, inv, now.w, mass) : make_float4(0.f, 0.f, 0.f, 0.f);
                }
                coef = live ? now.w * L.scale : 0.0f;
            } else {
                m = now.st.x;
                inv = now.st.y;
                mass = now.st.w;
                coef = now.st.z * up * L.scale;
            }
            a = live ? coef * mass * inv : 0.0f;
        } else {
            float hot = 0.0f;
            if (kStat) {
                const float lp = live ? (zy - m) * L.scale - log_s : 0.0f;
                float2 h = make_float2(0.0f, 0.0f);
                if (kHead == kHeadPolicy && live) {
                    h = policy_head(L, lp, old_logp, adv, ref);
                    h.y *= now.w;
                }
                if (lane == 0) {
                    if (kHead == kHeadPolicy) {
                        L.row_loss[r] = h.x;
                        L.row_logp[r] = lp;
                    }
                    if (L.state) L.state[r] = live ? make_float4(m, inv, lp, h.y) : make_float4(0.f, 0.f, 0.f, 0.f);
                }
                hot = h.y * L.scale;
            } else {
                m = now.st.x;
                inv = now.st.y;
                hot = now.st.w * up * L.scale;
            }
            a = -hot * inv;
            at_target = target_gradient(zy, m, a, hot, c);
        }
        if (!kGrad) continue;
        const bool aligned = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
        const auto element = [&](float x, int i) {
            float g = a * ex2((x - m) * c);
            if (kDistill) g -= coef * dense[i];
            else if (i == now.y) g = at_target;
            return g;
        };
#pragma unroll
        for (int h = 0; h < kN; ++h) {
            const int at = head + (lane + 32 * h) * kV;
            if (lane + 32 * h >= n) break;
            float2 x[kP];
            if (live) {
                Granule<T>::widen(u[h], x);
#pragma unroll
                for (int j = 0; j < kP; ++j) x[j] = make_float2(element(x[j].x, at + 2 * j), element(x[j].y, at + 2 * j + 1));
            } else {
#pragma unroll
                for (int j = 0; j < kP; ++j) x[j] = make_float2(0.0f, 0.0f);
            }
            const uint4 g = Granule<T>::narrow(x);
            if (aligned) *reinterpret_cast<uint4*>(out + at) = g;
            else store_elements<T>(out + at, &g);
        }
        if (loose >= 0) out[loose] = from_f32<T>(live ? element(loose_z, loose) : 0.0f);
        __syncwarp();  // before the next row's teacher
    }
    if (L.sum_out && blockIdx.x == 0) {  // a loss to add up: of these rows (by the only block), or given
        const float* value = kStat ? L.row_loss : L.sum_value;
        const float* weight = kStat ? L.weight : L.sum_weight;
        const int64_t n = kStat ? L.rows : L.sum_n;
        __syncthreads();
        const Sum2 s = weighted_sum(value, weight, n, threadIdx.x, blockDim.x);
        if (lane == 0) part[warp] = s;
        __syncthreads();
        if (warp == 0) {
            Sum2 t;
            if (lane < warps) t = part[lane];
            t.reduce();
            if (lane == 0) *L.sum_out = static_cast<float>(mean_of(t.value(), weight, n));
        }
    }
}

template <typename T, int kHead, int kForm>
cudaError_t launch_short(LossRows L, bool* summed, cudaStream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    // Few rows: one block of 32 warps takes them all and adds up the loss, which
    // saves a launch; it costs two rows a warp in turn at most.
    const bool alone = kForm != kBwd && L.sum_out && L.rows <= 64;
    if (kForm != kBwd && !alone) L.sum_out = nullptr;
    if (summed) *summed = alone;
    const int threads = alone ? 1024 : 256;
    const int64_t warps = threads / 32, most = device_info(dev).sm_count * int64_t(8);
    const int64_t blocks = (L.rows + warps - 1) / warps;
    const size_t smem = kHead == kHeadDistill && kForm != kFwd ? static_cast<size_t>(warps) * L.cols * 4 : 0;
    auto kernel = loss_short_kernel<T, kHead, kForm>;
    // The limit belongs to the function, whoever calls it: always the most that any call needs.
    constexpr size_t most_smem = 32 * (kShortBytes / sizeof(T)) * 4;
    if (smem > 48 * 1024) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most_smem));
        if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc = {};
    lc.gridDim = dim3(static_cast<unsigned>(alone ? 1 : blocks < most ? blocks : most));
    lc.blockDim = dim3(static_cast<unsigned>(threads));
    lc.dynamicSmemBytes = smem;
    lc.stream = stream;
    lc.attrs = &attr;
    lc.numAttrs = 1;
    return cudaLaunchKernelEx(&lc, kernel, L);
}

}  // namespace loss
}  // namespace lik
