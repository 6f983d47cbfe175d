// loss_rows.cuh -- the row kernel of the training objectives: softmax
// statistics, loss head and gradient of a row of logits that stays on chip
// between its two passes.
//
// A row is split into slices over the CTAs of a cluster.  In each CTA
//   - the loader (one warp) streams the slice's 16-byte granules into a ring
//     of shared-memory chunks (cp.async.bulk);
//   - the consumers walk the chunks for the max and the sum of exponentials,
//     and every warp sends its pair to the cluster's first CTA;
//   - there the closer (one warp) merges them, computes the loss head and
//     sends every CTA what the gradient needs: the max and the coefficients;
//   - the consumers walk the same chunks again and turn the logits into the
//     gradient where they lie;
//   - the storer (one warp) writes the chunks out (cp.async.bulk) and hands
//     them back to the loader.
// So a step reads a row from memory once and writes its gradient once, and
// loads, arithmetic and stores of neighbouring rows overlap.  (Stored by the
// consumers' own instructions the gradient held them up: every later shared
// memory access queued behind the stores.)  For distillation one more warp,
// the teacher's, prepares the entries of the next row (probabilities, the
// student's logits at their columns); the storer writes the row's loss and
// puts the gradient at the teacher's columns right before it stores a chunk.
//
// Rows that are left out, or whose gradient is known to be zero, are not
// read.  Each warp looks at 32 rows at a time, one a lane, to know which.
//
// Rows start at any element address: the granules are the aligned 16-byte
// words inside the row; the few elements before and after them are handled
// one by one by the first CTA of the cluster.
//
// Every wait is bounded.  Statistics and coefficients travel as st.async
// messages counted by mbarriers, in buffers of four rows; the comments at the
// barriers say why none is overwritten before it is read.
//
// Memory bounds it: a step moves 2 x 64 KB of a row per SM in 11,000 cycles, as
// a copy kernel does.  What it loses against a copy of the same bytes is its
// start and end (some 10 us with the sum's launch), the clusters' last round,
// and that SMs get unequal shares of the memory's rate (the mean SM is done
// at 0.88 of the slowest's time).  Measured (events, inputs beyond L2, with the
// sum) bf16: distillation step of 4096 x 128000 371 us where its bytes take 309;
// policy step of 8192 x 64000, a quarter of the rows left out, 299 us (271).
// The same step as a forward and a backward reads the logits twice: 1.5 times
// these bytes.
#pragma once

#include <atomic>

#include "dtype_load.cuh"
#include "lik_internal.h"
#include "losses.h"
#include "loss_math.cuh"
#include "sm100_ptx.cuh"

namespace lik {
namespace loss {

constexpr int kMaxSlots = 8;
constexpr int kMaxCluster = 8;
constexpr int kMaxWarps = 8;
constexpr int kMinSliceBytes = 4096;  // a row is not split finer for want of rows
constexpr int kSideWarps = 4;         // loader, closer, storer, teacher
constexpr int kPlanRows = 1 << 14;    // rows that are dealt out evenly by what they cost (3 KB of shared memory)
constexpr int kZeros = 128;           // granules of zeros that rows left out are stored from

// Shared memory of a CTA when `ctas` share an SM's 228 KB (1 KB each is taken).
constexpr size_t ring_smem(int ctas) { return static_cast<size_t>(228 / ctas - 1) * 1024; }

struct RingConfig {
    int cluster;       // CTAs per row
    int slots;         // ring chunks, of kNG granules per consumer thread
    int hold;          // chunks of a row that stay in the ring between a step's two passes, at most
    int k_pad;         // teacher entries, rounded up (distillation)
    int filter_words;  // of each of the two bit sets that find duplicate columns
    int planned;       // deal rows out by a plan
};

// ------------------------------------------------------- PTX not shared --

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync_all() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
// Messages to another CTA's shared memory, counted by an mbarrier there: no
// fence is needed on either side.
__device__ __forceinline__ void send(uint32_t to, float2 v, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1, %2}, [%3];" ::"r"(to),
                 "f"(v.x), "f"(v.y), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void send(uint32_t to, float4 v, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
                 "f"(v.x), "f"(v.y), "f"(v.z), "f"(v.w), "r"(bar)
                 : "memory");
}
// Bounded wait of a thread that, once one has run out, waits no more but goes
// through the rest of its work (on rubbish): the warps stay together, every
// collective is reached, and the kernel ends.  The error word tells the host.
// The slow part is not inlined: the row loop's code should stay in the
// instruction cache of an SM's quarter.
static __device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, unsigned int* err, unsigned ns) {
    return ns ? ptx::mbar_wait_nap(bar, parity, err, ns) : ptx::mbar_wait(bar, parity, err);
}
__device__ __forceinline__ void wait(uint64_t* bar, uint32_t parity, bool& late, unsigned int* err) {
    if (!ptx::mbar_test_wait(ptx::smem_u32(bar), parity) && !late) late = !wait_slow(ptx::smem_u32(bar), parity, err, 0);
}
// The same, asleep between its tests: a warp that polls takes issue slots from
// the warps it waits for.
__device__ __forceinline__ void wait_nap(uint64_t* bar, uint32_t parity, bool& late, unsigned int* err) {
    if (!ptx::mbar_test_wait(ptx::smem_u32(bar), parity) && !late) late = !wait_slow(ptx::smem_u32(bar), parity, err, 50);
}
__device__ __forceinline__ void bulk_prefetch(const void* src, uint32_t bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(src), "r"(bytes) : "memory");
}
// The other way, into the thread's current bulk group.
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// All but the thread's last kLeft groups have read their shared memory.
template <int kLeft>
__device__ __forceinline__ void bulk_wait_read() {
    asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kLeft) : "memory");
}
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
// This thread's shared-memory accesses come before bulk copies issued after a barrier.
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// `bytes` (a multiple of 16) from a 16-byte aligned global address.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
        "l"(src), "r"(bytes), "r"(bar)
        : "memory");
}

// ------------------------------------------------------- row geometry --

// The 16-byte granules inside a row and this CTA's share of them.
template <typename T>
struct Slice {
    int head;        // elements before the first granule
    int tail_at;     // first element after the last granule
    int first, n;    // granules [first, first + n) of the row
    __device__ Slice(const T* row, int cols, uint32_t rank, int cluster) {
        constexpr int kV = 16 / sizeof(T);
        const int skew = static_cast<int>((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
        head = skew ? kV - skew : 0;
        if (head > cols) head = cols;
        const int granules = (cols - head) / kV;
        tail_at = head + granules * kV;
        const int per = (granules + cluster - 1) >> (31 - __clz(cluster));  // a power of two
        first = static_cast<int>(rank) * per;
        if (first > granules) first = granules;
        n = granules - first < per ? granules - first : per;
    }
};

// A step's two passes over the n chunks of a slice: the first takes them in
// order and hands back all but the last `kept`; the second takes those, then the
// others from the last to the first (those read last are the likeliest in L2).
// The ring positions of the second pass follow each other.
struct Passes {
    int n, kept;
    __device__ Passes(int granules, int chunk, int hold) {
        n = (granules + chunk - 1) / chunk;
        kept = n < hold ? n : hold;
    }
    __device__ int second(int k) const { return k < kept ? n - kept + k : n - 1 - k; }
};

// The element outside the granules that this thread owns, or -1: threads 0..
// take the head, threads 32.. the tail, in the first CTA.
template <typename T>
__device__ __forceinline__ int loose_element(const Slice<T>& s, int cols, uint32_t rank, int tid) {
    if (rank != 0) return -1;
    if (tid < s.head) return tid;
    if (tid >= 32 && tid - 32 < cols - s.tail_at) return s.tail_at + tid - 32;
    return -1;
}

// -------------------------------------------------------- shared memory --

constexpr int kBuf = 4;  // rows that messages are buffered for

// Control words, behind the ring; the teacher's entries follow them.  Rows
// are counted by j among the rows that are read; buffer j % 4.
struct Control {
    // A chunk is loaded; the consumers have its gradient (forms with one) or are
    // done with it; the loader may refill it.
    uint64_t full[kMaxSlots], done[kMaxSlots], empty[kMaxSlots];
    // First CTA: the pairs of every warp of the cluster.  With a gradient a
    // consumer sends row j's after its CTA's storer closed row j - 4 and it has had
    // go of row j - 1; without one, after go of row j - 3: the closer has used row
    // j - 4's either way.
    uint64_t stat[kBuf];
    float2 parts[kBuf][kMaxCluster * kMaxWarps];
    // First CTA: the teacher mass from every CTA's teacher warp, sent for row j
    // after the storer freed row j - 2's entries, and so had go of it.
    uint64_t ready[kBuf];
    float2 mass[kBuf][kMaxCluster];
    // Every CTA: (max, coefficient of e, the gradient at the target or the sum,
    // the row's weight) from the closer.
    uint64_t go[kBuf];
    float4 verdict[kBuf];
    // Every CTA: the storer is done with row j, and so with its verdict; consumers
    // send row j + 4's pairs after that.
    uint64_t closed[kBuf];
    // Every CTA, between its teacher's warp (row j's entries are in buffer j % 2)
    // and the storer (it is done with them).
    uint64_t prepared[2], freed[2];
};

// Waits (bounded) for this CTA's last copies, so that none lands in shared
// memory the kernel no longer holds: at once, unless another wait ran out.
static __device__ __noinline__ void drain(Control* ctl, int slots, int slot, uint32_t phase, unsigned int* err) {
    for (int i = 0; i < slots; ++i) {
        // the slot's last load was of this trip (before `slot`) or of the one before
        const uint32_t last = i < slot ? phase : phase ^ 1;
        if (!ptx::mbar_wait(ptx::smem_u32(&ctl->full[i]), last, err)) return;
    }
}

__device__ __forceinline__ void arrive(uint64_t* bar) { ptx::mbar_arrive(ptx::smem_u32(bar)); }
__device__ __forceinline__ void expect(uint64_t* bar, uint32_t bytes) {
    ptx::mbar_arrive_expect_tx(ptx::smem_u32(bar), bytes);
}

// Which rows are read, for up to kPlanRows of them: rows are dealt out to the
// clusters in turn, first those that are read, then the others, so that every
// cluster gets its share of the work however the mask lies.
struct Plan {
    uint32_t bits[kPlanRows / 32];    // row 32 w + i is read: bit i of word w
    uint16_t before[kPlanRows / 32];  // rows read before word w
    int read;                         // rows read
};

// Fills the plan (all threads of the CTA, a multiple of 32).
template <int kHead, bool kStat>
__device__ void make_plan(Plan* plan, const LossRows& L) {
    constexpr int kBatch = 8;
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5, words = static_cast<int>((L.rows + 31) / 32);
    for (int w0 = threadIdx.x >> 5; w0 < words; w0 += kBatch * warps) {
        Peek p[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) p[i] = peek<kHead, kStat>(L, static_cast<int64_t>(w0 + i * warps) * 32 + lane);
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int w = w0 + i * warps;
            const uint32_t b = __ballot_sync(0xffffffffu, static_cast<int64_t>(w) * 32 + lane < L.rows && is_read<kHead, kStat>(L, p[i]));
            if (lane == 0 && w < words) plan->bits[w] = b;
        }
    }
    __syncthreads();
    if (threadIdx.x < 32) {
        const int each = (words + 31) / 32, from = lane * each, to = min(words, from + each);
        int n = 0;
        for (int w = from; w < to; ++w) n += __popc(plan->bits[w]);
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o *= 2) {
            const int v = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += v;
        }
        if (lane == 31) plan->read = sum;
        sum -= n;
        for (int w = from; w < to; ++w) {
            plan->before[w] = static_cast<uint16_t>(sum);
            sum += __popc(plan->bits[w]);
        }
    }
    __syncthreads();
}

// The o-th row of the plan's order, 0 <= o < rows.
static __device__ __noinline__ int64_t planned_row(const Plan* plan, int64_t rows, int64_t o) {
    const bool read = o < plan->read;
    const int k = static_cast<int>(read ? o : o - plan->read);
    int lo = 0, hi = static_cast<int>((rows + 31) / 32) - 1;  // the last word with at most k such rows before it
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        const int n = read ? plan->before[mid] : mid * 32 - plan->before[mid];
        if (n <= k) lo = mid;
        else hi = mid - 1;
    }
    uint32_t b = read ? plan->bits[lo] : ~plan->bits[lo];
    for (int i = k - (read ? plan->before[lo] : lo * 32 - plan->before[lo]); i > 0; --i) b &= b - 1;
    return lo * 32 + __ffs(b) - 1;
}

// A warp's walk over its cluster's rows, 32 at a time, one a lane, the next 32
// loaded ahead.
template <int kHead, bool kStat>
struct Walk {
    const LossRows& L;
    const Plan* plan;  // nullptr: rows in their own order
    int64_t step, base;
    int lane;
    int64_t row, row_ahead;  // this lane's
    Peek mine, ahead;
    uint32_t live = 0;  // bit i: lane i's row is read
    int n = 0;          // rows of this batch

    __device__ __forceinline__ Walk(const LossRows& rows, const Plan* order, int64_t first, int64_t stride, int lane_)
        : L(rows), plan(order), step(stride), base(first), lane(lane_) {
        look(base);
        load();
    }
    __device__ __forceinline__ void look(int64_t from) {
        int64_t o = from + lane * step;
        if (!kStat && o < L.rows) {
            // Backwards: the rows a forward read last are the likeliest in L2.
            const int64_t read = plan ? plan->read : L.rows;
            if (o < read) o = read - 1 - o;
        }
        row_ahead = plan && o < L.rows ? planned_row(plan, L.rows, o) : o;
        ahead = peek<kHead, kStat>(L, row_ahead);
    }
    __device__ __forceinline__ void load() {
        mine = ahead;
        row = row_ahead;
        look(base + 32 * step);
        live = __ballot_sync(0xffffffffu, row < L.rows && is_read<kHead, kStat>(L, mine));
        const int64_t left = base < L.rows ? (L.rows - base + step - 1) / step : 0;
        n = left < 32 ? static_cast<int>(left) : 32;
    }
    __device__ __forceinline__ void advance() {
        base += 32 * step;
        load();
    }
    __device__ __forceinline__ int64_t at(int i) const { return __shfl_sync(0xffffffffu, row, i); }
    __device__ __forceinline__ float from(float v, int i) const { return __shfl_sync(0xffffffffu, v, i); }
    __device__ __forceinline__ int target(int i) const { return __shfl_sync(0xffffffffu, mine.y, i); }
};

// ------------------------------------------------------------ the kernel --

template <typename T, int kHead, int kForm, int kWarps, int kNG>
__global__ void __launch_bounds__(kWarps * 32 + kSideWarps * 32)
    loss_ring_kernel(const LossRows L, const RingConfig cfg, unsigned int* err) {
    constexpr int kV = 16 / sizeof(T);
    constexpr int kNT = kWarps * 32;
    constexpr int kChunk = kNT * kNG;  // granules per chunk
    constexpr bool kDistill = kHead == kHeadDistill;
    constexpr bool kGrad = kForm != kFwd;
    constexpr bool kStat = kForm != kBwd;
    constexpr bool kGo = kStat || kDistill;  // the closer decides a row; else its saved state does
    extern __shared__ __align__(128) unsigned char smem[];
    uint4* ring = reinterpret_cast<uint4*>(smem);
    uint4* zeros = ring + cfg.slots * kChunk;  // kZeros granules, with a gradient
    Control* ctl = reinterpret_cast<Control*>(zeros + (kGrad ? kZeros : 0));
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t rank = cluster_rank();
    const int cols = static_cast<int>(L.cols);
    const int64_t step = gridDim.x / cfg.cluster;  // clusters; rows are dealt out in turn
    const int64_t first_row = blockIdx.x / cfg.cluster;
    const float c = L.c;
    const T* logits = static_cast<const T*>(L.logits);

    if (tid == 0) {
        for (int i = 0; i < cfg.slots; ++i) {
            ptx::mbar_init(ptx::smem_u32(&ctl->full[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&ctl->done[i]), kWarps);
            ptx::mbar_init(ptx::smem_u32(&ctl->empty[i]), kGrad ? 1 : kWarps);
        }
        for (int i = 0; i < kBuf; ++i) {
            ptx::mbar_init(ptx::smem_u32(&ctl->stat[i]), kWarps + (cfg.cluster > 1 ? 1 : 0));
            ptx::mbar_init(ptx::smem_u32(&ctl->ready[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&ctl->go[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&ctl->closed[i]), 1);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(ptx::smem_u32(&ctl->prepared[i]), 1);
            ptx::mbar_init(ptx::smem_u32(&ctl->freed[i]), 1);
        }
        ptx::fence_mbar_init();
    }
    if (kGrad) {
        for (int i = tid; i < kZeros; i += blockDim.x) zeros[i] = make_uint4(0, 0, 0, 0);
        fence_async();
    }
    cluster_sync_all();
    grid_launch_dependents();
    grid_wait();
    Plan* plan = nullptr;
    if (cfg.planned) {
        plan = reinterpret_cast<Plan*>(reinterpret_cast<unsigned char*>(ctl + 1) +
                                       (kDistill ? Entries::bytes(cfg.k_pad, cfg.filter_words) : 0));
        make_plan<kHead, kStat>(plan, L);
    }

    if (warp == kWarps) {
        // ---------------------------------------------------- the loader --
        // Besides loading a row it asks L2 for the next one: the ring cannot hold it,
        // and its loads should not wait for memory once there is room.
        int slot = 0;
        uint32_t phase = 0;
        bool ok = true;
        const auto load = [&](const T* from, int g, int n) {
            const uint32_t bytes = static_cast<uint32_t>(n - g < kChunk ? n - g : kChunk) * 16;
            bool late = !ok;
            wait_nap(&ctl->empty[slot], phase ^ 1, late, err);
            ok = !late;
            if (!ok) return;
            expect(&ctl->full[slot], bytes);
            bulk_load(ptx::smem_u32(ring + slot * kChunk), from + static_cast<int64_t>(g) * kV, bytes,
                      ptx::smem_u32(&ctl->full[slot]));
            if (++slot == cfg.slots) slot = 0, phase ^= 1;
        };
        for (Walk<kHead, kStat> w(L, plan, first_row, step, lane); ok && w.n > 0; w.advance()) {
            for (uint32_t todo = w.live; todo; todo &= todo - 1) {
                const uint32_t more = todo & (todo - 1);
                const int64_t r = w.at(__ffs(todo) - 1), r_next = w.at(more ? __ffs(more) - 1 : 0);
                if (lane == 0 && ok) {
                    const T* row = logits + r * L.stride;
                    const Slice<T> s(row, cols, rank, cfg.cluster);
                    const T* from = row + s.head + static_cast<int64_t>(s.first) * kV;
                    const Passes t(s.n, kChunk, cfg.hold);
                    for (int k = 0; k < t.n; ++k) load(from, k * kChunk, s.n);
                    if (kForm == kStep) {
                        if (more) {
                            const T* next = logits + r_next * L.stride;
                            const Slice<T> f(next, cols, rank, cfg.cluster);
                            if (f.n > 0)
                                bulk_prefetch(next + f.head + static_cast<int64_t>(f.first) * kV,
                                              static_cast<uint32_t>(f.n) * 16);
                        }
                        for (int k = t.kept; k < t.n; ++k) load(from, t.second(k) * kChunk, s.n);
                    }
                }
                __syncwarp();
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        }
        if (lane == 0) drain(ctl, cfg.slots, slot, phase, err);
    } else if (warp == kWarps + 1) {
        // ---------------------------------------------------- the closer --
        if (!kGo && L.sum_out && blockIdx.x == 0) {  // the loss that this gradient belongs to
            const Sum2 sum = weighted_sum(L.sum_value, L.sum_weight, L.sum_n, lane, 32);
            if (lane == 0) *L.sum_out = static_cast<float>(mean_of(sum.value(), L.sum_weight, L.sum_n));
        }
        if (kGo && rank == 0) {
            const float up = kForm == kBwd && L.grad_loss ? *L.grad_loss : 1.0f;
            bool late = false;
            int j = 0;
            for (Walk<kHead, kStat> w(L, plan, first_row, step, lane); w.n > 0; w.advance()) {
                // what the head needs of 32 rows
                const int64_t mine = w.row;
                float zy = 0.0f, old_logp = 0.0f, adv = 0.0f, ref = 0.0f;
                if (!kDistill && (w.live >> lane & 1)) {
                    zy = load_f32(logits + mine * L.stride + w.mine.y);
                    if (kHead == kHeadPolicy) {
                        old_logp = L.old_logp[mine];
                        adv = L.advantage[mine];
                        if (L.ref_logp) ref = L.ref_logp[mine];
                    }
                }
                if (!kDistill && lane < w.n && !(w.live >> lane & 1)) {  // rows left out
                    if (kHead == kHeadPolicy) {
                        L.row_loss[mine] = 0.0f;
                        L.row_logp[mine] = 0.0f;
                    }
                    if (L.state) L.state[mine] = make_float4(0.f, 0.f, 0.f, 0.f);
                }
                for (uint32_t todo = w.live; todo; todo &= todo - 1, ++j) {
                    const int i = __ffs(todo) - 1, b = j % kBuf;
                    const uint32_t phase = (j / kBuf) & 1;
                    const int64_t r = w.at(i);
                    const float weight = w.from(w.mine.w, i);
                    float4 v;
                    if (kStat) {
                        wait(&ctl->stat[b], phase, late, err);
                        Stat total = {-INFINITY, 0.0f};
                        if (lane < kWarps * cfg.cluster) total = {ctl->parts[b][lane].x, ctl->parts[b][lane].y};
                        for (int k = lane + 32; k < kWarps * cfg.cluster; k += 32) {
                            const float2 p = ctl->parts[b][k];
                            const float m = fmaxf(total.m, p.x), o = offset_of(m);
                            total = {m, total.s * ex2((total.m - o) * c) + p.y * ex2((p.x - o) * c)};
                        }
                        total = warp_merge(total, c);
                        const bool live = total.s != 0.0f;
                        const float m = offset_of(total.m), inv = live ? 1.0f / total.s : 0.0f;
                        if (kDistill) {
                            wait(&ctl->ready[b], phase, late, err);
                            const float mass = ctl->mass[b][0].x;
                            v = make_float4(m, live && mass != 0.0f ? weight * L.scale * mass * inv : 0.0f, total.s, weight);
                        } else {
                            const float zt = w.from(zy, i), lp = live ? (zt - m) * L.scale - logf(total.s) : 0.0f;
                            float2 h = make_float2(0.0f, 0.0f);
                            if (kHead == kHeadPolicy) {
                                const float o = w.from(old_logp, i), a = w.from(adv, i), q = w.from(ref, i);
                                if (live) h = policy_head(L, lp, o, a, q);
                                h.y *= weight;
                            }
                            if (lane == 0) {
                                if (kHead == kHeadPolicy) {
                                    L.row_loss[r] = h.x;
                                    L.row_logp[r] = lp;
                                }
                                if (L.state) L.state[r] = make_float4(m, inv, lp, h.y);
                            }
                            const float hot = h.y * L.scale;
                            v = make_float4(m, -hot * inv, target_gradient(zt, m, -hot * inv, hot, c), 0.0f);
                        }
                    } else {  // distillation from its saved state: (max, 1 / sum, weight, mass)
                        wait(&ctl->ready[b], phase, late, err);
                        const float st_w = w.from(w.mine.st.z, i) * up;
                        v = make_float4(w.from(w.mine.st.x, i),
                                        st_w * L.scale * w.from(w.mine.st.w, i) * w.from(w.mine.st.y, i), 1.0f, st_w);
                    }
                    if (lane == 0) {
                        ctl->verdict[b] = v;
                        arrive(&ctl->go[b]);
                    } else if (lane < cfg.cluster) {
                        send(map_rank(ptx::smem_u32(&ctl->verdict[b]), lane), v, map_rank(ptx::smem_u32(&ctl->go[b]), lane));
                    }
                }
            }
        }
    } else if (warp == kWarps + 2) {
        // ---------------------------------------------------- the storer --
        if (kGrad || kDistill) {
            const Entries e(ctl + 1, cfg.k_pad, cfg.filter_words);
            const float up = !kGo && L.grad_loss ? *L.grad_loss : 1.0f;
            int slot = 0, j = 0, unread = -1;  // unread: the slot whose store may still read it
            uint32_t phase = 0;
            bool late = false;
            // The slot stored last is handed back with the next store, or before the storer
            // waits for anything: the loader may need it first.
            const auto hand_back = [&] {
                if (unread >= 0 && lane == 0) {
                    bulk_wait_read<0>();
                    arrive(&ctl->empty[unread]);
                }
                unread = -1;
            };
            const auto await = [&] {
                if (!ptx::mbar_test_wait(ptx::smem_u32(&ctl->done[slot]), phase)) hand_back();
                wait_nap(&ctl->done[slot], phase, late, err);
                __syncwarp();
            };
            for (Walk<kHead, kStat> w(L, plan, first_row, step, lane); w.n > 0; w.advance()) {
                if (kDistill && kStat && rank == 0 && lane < w.n && !(w.live >> lane & 1)) left_out(L, w.row);
                for (int q = 0; q < w.n; ++q) {
                    const int64_t r = w.at(q);
                    T* out = kGrad ? static_cast<T*>(L.grad) + r * L.grad_stride : nullptr;
                    if (!(w.live >> q & 1)) {
                        if (!kGrad) continue;
                        const Slice<T> s(out, cols, rank, cfg.cluster);
                        if (lane == 0) {
                            for (int g = 0; g < s.n; g += kZeros)
                                bulk_store(out + s.head + static_cast<int64_t>(s.first + g) * kV, ptx::smem_u32(zeros),
                                           static_cast<uint32_t>(s.n - g < kZeros ? s.n - g : kZeros) * 16);
                            bulk_commit();
                        }
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int i = loose_element(s, cols, rank, lane + 32 * h);
                            if (i >= 0) out[i] = from_f32<T>(0.0f);
                        }
                        continue;
                    }
                    const T* z = logits + r * L.stride;
                    const Slice<T> s(z, cols, rank, cfg.cluster);
                    const int buf = j & 1, b = j % kBuf;
                    const Passes t(s.n, kChunk, cfg.hold);
                    if (kForm == kStep) {  // chunks of the statistics pass that do not stay
                        for (int k = t.kept; k < t.n; ++k) {
                            await();
                            if (lane == 0) arrive(&ctl->empty[slot]);
                            if (++slot == cfg.slots) slot = 0, phase ^= 1;
                        }
                    }
                    float4 v;
                    if (kGo) {
                        hand_back();
                        wait_nap(&ctl->go[b], (j / kBuf) & 1, late, err);
                        v = ctl->verdict[b];
                    } else {
                        const float hot = w.from(w.mine.st.w, q) * up * L.scale;
                        v.x = w.from(w.mine.st.x, q);
                        v.y = -hot * w.from(w.mine.st.y, q);
                        v.z = target_gradient(load_f32(z + w.target(q)), v.x, v.y, hot, c);
                    }
                    const float m = v.x;
                    const int* index = e.index + buf * e.pad;
                    const float *p = e.p + buf * e.pad, *x = e.z + buf * e.pad;
                    Teacher sums = {0.0f, 0.0f, 0.0f};
                    bool any = false;  // the row has a gradient and a loss
                    // this lane's first entries: column and gradient there (later ones are worked out as they are met)
                    constexpr int kOwn = 4;
                    int own_i[kOwn];
                    float own_g[kOwn];
                    const float coef = kDistill ? v.w * L.scale : 0.0f;
                    const auto entry_gradient = [&](int k) { return v.y * ex2((x[k] - m) * c) - coef * p[k]; };
                    if (kDistill) {
                        wait(&ctl->prepared[buf], (j >> 1) & 1, late, err);
                        __syncwarp();
                        sums = e.sums[buf];
                        any = v.z != 0.0f && sums.mass != 0.0f;
                        if (kGrad)
#pragma unroll
                            for (int h = 0; h < kOwn; ++h) {
                                const bool in = any && lane + 32 * h < L.k;
                                own_i[h] = in ? index[lane + 32 * h] : -1;
                                own_g[h] = in ? entry_gradient(lane + 32 * h) : 0.0f;
                            }
                    }
                    if (kGrad) {
                        const bool aligned = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
                        const int lo = s.head + s.first * kV;  // first element of the slice's granules
                        const int y = kDistill ? -1 : w.target(q);
                        // the elements outside the granules: the head, then the tail
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int i = loose_element(s, cols, rank, lane + 32 * h);
                            if (i < 0) continue;
                            out[i] = from_f32<T>(!kDistill && i == y ? v.z : v.y * ex2((load_f32(z + i) - m) * c));
                        }
                        if (kDistill && any && rank == 0 && (s.head > 0 || s.tail_at < cols)) {
                            __syncwarp();
                            for (int k = lane; k < L.k; k += 32) {
                                const int i = index[k];
                                if (i >= 0 && (i < s.head || i >= s.tail_at)) out[i] = from_f32<T>(entry_gradient(k));
                            }
                        }
                        for (int k = 0; k < t.n; ++k) {
                            const int g = (kForm == kStep ? t.second(k) : k) * kChunk;
                            await();
                            const int n = s.n - g < kChunk ? s.n - g : kChunk, at = lo + g * kV;
                            T* chunk = reinterpret_cast<T*>(ring + slot * kChunk);
                            if (!kDistill && static_cast<unsigned>(y - at) < static_cast<unsigned>(n * kV)) {
                                if (lane == 0) (aligned ? chunk : out + at)[y - at] = from_f32<T>(v.z);
                                fence_async();
                            }
                            if (kDistill && any) {
                                T* to = aligned ? chunk : out + at;
                                const unsigned size = static_cast<unsigned>(n * kV);
                                bool wrote = false;
#pragma unroll
                                for (int h = 0; h < kOwn; ++h) {
                                    const int i = own_i[h] - at;
                                    if (own_i[h] >= 0 && static_cast<unsigned>(i) < size) to[i] = from_f32<T>(own_g[h]), wrote = true;
                                }
                                for (int o = lane + 32 * kOwn; o < L.k; o += 32) {
                                    const int i = index[o] - at;
                                    if (index[o] >= 0 && static_cast<unsigned>(i) < size)
                                        to[i] = from_f32<T>(entry_gradient(o)), wrote = true;
                                }
                                if (wrote) fence_async();
                                __syncwarp();
                            }
                            if (lane == 0) {
                                if (aligned) {
                                    bulk_store(out + at, ptx::smem_u32(chunk), n * 16);
                                    bulk_commit();
                                    if (unread >= 0) {
                                        bulk_wait_read<1>();
                                        arrive(&ctl->empty[unread]);
                                    }
                                } else {
                                    arrive(&ctl->empty[slot]);
                                }
                            }
                            if (aligned) unread = slot;
                            if (++slot == cfg.slots) slot = 0, phase ^= 1;
                        }
                    }
                    if (kDistill && kStat && rank == 0) {
                        const float loss = any ? teacher_loss(L, e, buf, sums, m, logf(v.z), lane) : 0.0f;
                        if (lane == 0) {
                            L.row_loss[r] = loss;
                            if (L.state)
                                L.state[r] = any ? make_float4(m, 1.0f / v.z, v.w, sums.mass) : make_float4(0.f, 0.f, 0.f, 0.f);
                        }
                    }
                    __syncwarp();
                    if (lane == 0) {
                        if (kDistill) arrive(&ctl->freed[buf]);
                        if (kGo) arrive(&ctl->closed[b]);
                    }
                    ++j;
                }
            }
            if (lane == 0) bulk_wait_all();
        }
    } else if (warp == kWarps + 3) {
        // ------------------------------------------------ the teacher's warp --
        if (kDistill) {
            const Entries e(ctl + 1, cfg.k_pad, cfg.filter_words);
            for (int i = lane; i < e.words; i += 32) e.seen[i] = 0, e.twice[i] = 0;
            __syncwarp();
            bool late = false;
            int j = 0;
            for (Walk<kHead, kStat> w(L, plan, first_row, step, lane); w.n > 0; w.advance()) {
                for (uint32_t todo = w.live; todo; todo &= todo - 1, ++j) {
                    const int buf = j & 1, b = j % kBuf;
                    if (j >= 2) wait_nap(&ctl->freed[buf], ((j >> 1) - 1) & 1, late, err);
                    const Teacher t = prepare_teacher<T>(L, w.at(__ffs(todo) - 1), e, buf, lane);
                    __syncwarp();
                    if (kGrad) merge_duplicates(e, buf, L.k, lane);
                    if (lane == 0) {
                        e.sums[buf] = t;
                        arrive(&ctl->prepared[buf]);
                        if (rank == 0) {
                            ctl->mass[b][0] = make_float2(t.mass, 0.0f);
                            expect(&ctl->ready[b], 8 * (cfg.cluster - 1));
                        } else {
                            send(map_rank(ptx::smem_u32(&ctl->mass[b][rank]), 0), make_float2(t.mass, 0.0f),
                                 map_rank(ptx::smem_u32(&ctl->ready[b]), 0));
                        }
                    }
                    __syncwarp();
                }
            }
        }
    } else {
        // -------------------------------------------------- the consumers --
        const float up = !kGo && L.grad_loss ? *L.grad_loss : 1.0f;
        int slot = 0, j = 0, q = 0;
        uint32_t phase = 0;
        bool late = false;
        Walk<kHead, kStat> w(L, plan, first_row, step, lane);
        while (true) {
            // the next row that is read
            bool have = false;
            int64_t r = 0;
            float m = 0.0f, a = 0.0f;  // the max; the coefficient of e
            while (w.n > 0) {
                if (q == w.n) {
                    w.advance();
                    q = 0;
                    continue;
                }
                if (w.live >> q & 1) {
                    r = w.at(q);
                    have = true;
                    break;
                }
                ++q;
            }
            if (!have) break;
            const T* z = logits + r * L.stride;
            const Slice<T> s(z, cols, rank, cfg.cluster);
            const Passes t(s.n, kChunk, cfg.hold);
            const int b = j % kBuf;
            const int loose = loose_element(s, cols, rank, tid);
            const float loose_z = kStat && loose >= 0 ? load_f32(z + loose) : 0.0f;
            if (kGo && tid == 0 && cfg.cluster > 1) {
                if (rank != 0) expect(&ctl->go[b], 16);
                else if (kStat) expect(&ctl->stat[b], kWarps * (cfg.cluster - 1) * 8);
            }
            if (!kGo) {
                m = w.from(w.mine.st.x, q);
                a = -w.from(w.mine.st.w, q) * up * L.scale * w.from(w.mine.st.y, q);
            }
            if (kStat) {
                Running v;
                int slot2 = slot;  // where the second pass starts
                uint32_t phase2 = phase;
                for (int k = 0; k < t.n; ++k) {
                    const int g = k * kChunk;
                    if (k == t.n - t.kept) slot2 = slot, phase2 = phase;
                    wait(&ctl->full[slot], phase, late, err);
                    const uint4* chunk = ring + slot * kChunk + tid;
                    uint4 u[kNG];
#pragma unroll
                    for (int h = 0; h < kNG; ++h) u[h] = chunk[h * kNT];
                    if (s.n - g < kChunk) {  // beyond the slice: logits of no weight
#pragma unroll
                        for (int h = 0; h < kNG; ++h)
                            if (tid + h * kNT >= s.n - g) u[h] = Granule<T>::nothing();
                    }
                    v.add_granules<T, kNG>(u, c);
                    if (kForm == kFwd || k < t.n - t.kept) {
                        __syncwarp();
                        if (lane == 0) arrive(kGrad ? &ctl->done[slot] : &ctl->empty[slot]);
                    }
                    if (++slot == cfg.slots) slot = 0, phase ^= 1;
                }
                if (loose >= 0) v.add(loose_z, c);
                const Stat total = warp_merge(v.stat(), c);
                if (kGrad && j >= kBuf) wait(&ctl->closed[b], (j / kBuf - 1) & 1, late, err);
                if (!kGrad && j >= 3) wait(&ctl->go[(j - 3) % kBuf], ((j - 3) / kBuf) & 1, late, err);
                if (lane == 0) {
                    float2* at = &ctl->parts[b][rank * kWarps + warp];
                    if (rank == 0) {
                        *at = make_float2(total.m, total.s);
                        arrive(&ctl->stat[b]);
                    } else {
                        send(map_rank(ptx::smem_u32(at), 0), make_float2(total.m, total.s),
                             map_rank(ptx::smem_u32(&ctl->stat[b]), 0));
                    }
                }
                if (kGrad) slot = slot2, phase = phase2;
            }
            if (kGrad) {
                T* out = static_cast<T*>(L.grad) + r * L.grad_stride;
                const bool aligned = ((reinterpret_cast<uintptr_t>(out) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
                if (kGo) {
                    // The row may be written (in place of the logits) from here on: whoever reads
                    // it elsewhere has done so before the closer could decide.
                    wait(&ctl->go[b], (j / kBuf) & 1, late, err);
                    const float4 v = ctl->verdict[b];
                    m = v.x;
                    a = v.y;
                }
                for (int k = 0; k < t.n; ++k) {
                    const int g = (kForm == kStep ? t.second(k) : k) * kChunk;
                    wait(&ctl->full[slot], phase, late, err);
                    uint4* chunk = ring + slot * kChunk + tid;
                    const int n = s.n - g - tid;  // what is left from this thread's granule on
                    uint4 u[kNG];
#pragma unroll
                    for (int h = 0; h < kNG; ++h) u[h] = gradient<T>(chunk[h * kNT], m, a, c);
#pragma unroll
                    for (int h = 0; h < kNG; ++h) chunk[h * kNT] = u[h];  // beyond the slice: of no use, and not stored
                    if (!aligned) {
                        T* to = out + s.head + static_cast<int64_t>(s.first + g + tid) * kV;
#pragma unroll 1
                        for (int i = 0; i < n && i < kChunk; i += kNT) store_elements<T>(to + i * kV, chunk + i);
                    }
                    fence_async();
                    __syncwarp();
                    if (lane == 0) arrive(&ctl->done[slot]);
                    if (++slot == cfg.slots) slot = 0, phase ^= 1;
                }
            }
            ++j;
            ++q;
        }
    }
    __syncwarp();
    cluster_sync_all();  // no CTA leaves while another may still send to it
}

// ------------------------------------------------------------ launching --

// CTAs that share a row.  In a step a slice has to fit what a CTA can hold
// between its two passes (`held` bytes; where even 8 CTAs do not, the rest is
// read again).  More than that pays where rows are few, or leave much idle in
// their last round: a round costs a CTA its slice's bytes at its share of an
// SM's 44 bytes a ns, and some 1.5 us of latency that the others' work does not
// cover, 0.8 more for each halving.  Rows in many rounds are best not split
// (8192 x 32000 bf16 in a step, 64 KB rows: 185 us by one CTA a row, 257 by two,
// 361 by four).
inline int pick_cluster(int64_t rows, int64_t row_bytes, int64_t held, int passes, int sm_count, int ctas) {
    int best = 0;
    double best_ns = 0.0;
    for (int c = 1; c <= kMaxCluster; c *= 2) {
        if (held > 0 && c < kMaxCluster && row_bytes > held * c) continue;
        if (best && row_bytes / c < kMinSliceBytes) break;
        const int64_t slots = static_cast<int64_t>(sm_count) * ctas / c;
        const double rounds = static_cast<double>((rows + slots - 1) / slots);
        const double wait = c == 1 ? 1500.0 : c == 2 ? 2300.0 : c == 4 ? 3100.0 : 3900.0;
        const double ns = rounds * (wait + static_cast<double>(row_bytes / c) * passes * ctas / 44.0);
        if (!best || ns < best_ns) best = c, best_ns = ns;
    }
    return best;
}

// How a CTA's shared memory is used; cluster is left open.
template <int kHead, int kForm, int kWarps, int kNG, int kCtas>
RingConfig ring_config(const LossRows& L, int sm_count) {
    RingConfig cfg;
    cfg.cluster = 1;
    cfg.k_pad = kHead == kHeadDistill ? (L.k + 31) / 32 * 32 : 0;
    cfg.filter_words = kHead == kHeadDistill ? filter_words(L.k) : 0;
    const bool masks = kHead != kHeadDistill || kForm == kBwd || L.weight;
    cfg.planned = masks && L.rows > sm_count && L.rows <= kPlanRows;
    const size_t fixed = sizeof(Control) + (kHead == kHeadDistill ? Entries::bytes(cfg.k_pad, cfg.filter_words) : 0) +
                         (cfg.planned ? sizeof(Plan) : 0) + (kForm == kFwd ? 0 : kZeros * 16);
    cfg.slots = fixed < ring_smem(kCtas) ? static_cast<int>((ring_smem(kCtas) - fixed) / (kWarps * 32 * 16 * kNG)) : 0;
    if (cfg.slots > kMaxSlots) cfg.slots = kMaxSlots;
    // one slot may still be being stored, and one is for the next chunk
    cfg.hold = kForm == kStep ? cfg.slots - 2 : 0;
    return cfg;
}

template <typename T, int kHead, int kForm, int kWarps, int kNG, int kCtas>
cudaError_t launch_ring(const LossRows& L, unsigned int* err, cudaStream_t stream) {
    constexpr int kChunkBytes = kWarps * 32 * 16 * kNG;
    constexpr int kThreads = (kWarps + kSideWarps) * 32;
    auto kernel = loss_ring_kernel<T, kHead, kForm, kWarps, kNG>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const DeviceInfo& info = device_info(dev);
    const size_t budget = ring_smem(kCtas);
    RingConfig cfg = ring_config<kHead, kForm, kWarps, kNG, kCtas>(L, info.sm_count);
    if (cfg.slots < 3) return cudaErrorInvalidConfiguration;
    cfg.cluster = pick_cluster(L.rows, L.cols * static_cast<int64_t>(sizeof(T)),
                               static_cast<int64_t>(cfg.hold) * kChunkBytes, kForm == kFwd ? 1 : 2, info.sm_count, kCtas);

    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim = {static_cast<unsigned>(cfg.cluster), 1, 1};
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t lc = {};
    lc.blockDim = dim3(kThreads);
    lc.dynamicSmemBytes = budget;
    lc.stream = stream;
    lc.attrs = attr;
    lc.numAttrs = 1;  // for the question about occupancy

    // clusters that run at once, per device and cluster size (0: not asked yet)
    static std::atomic<int> resident_clusters[64][4];
    const int log_c = cfg.cluster == 1 ? 0 : cfg.cluster == 2 ? 1 : cfg.cluster == 4 ? 2 : 3;
    std::atomic<int>& known = resident_clusters[dev % 64][log_c];
    int clusters = known.load();
    if (clusters == 0) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(budget));
        if (e != cudaSuccess) return e;
        lc.gridDim = dim3(cfg.cluster);
        e = cudaOccupancyMaxActiveClusters(&clusters, kernel, &lc);
        if (e != cudaSuccess) return e;
        if (clusters < 1) return cudaErrorLaunchOutOfResources;
        known.store(clusters);
    }
    const int64_t used = L.rows < clusters ? L.rows : clusters;
    lc.gridDim = dim3(static_cast<unsigned>(used * cfg.cluster));
    lc.numAttrs = 2;
    return cudaLaunchKernelEx(&lc, kernel, L, cfg, err);
}

}  // namespace loss
}  // namespace lik
