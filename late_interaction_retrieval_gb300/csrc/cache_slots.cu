// cache_slots.cu -- block tables and slot maps of a batch from its requests'
// lengths.
//
// Two prefix sums over the requests (new tokens, new pages) place everything
// else: a token's request is found in the first, a new page's request in the
// second.  Every block sums all requests for itself into its shared memory
// (12 bytes a request, from L2) and then fills its share of the slots and the
// table, so that one launch does it with no block waiting for another.  What
// bounds it is the work (62% of the issue slots, 60% of the ALU) and the chain
// of a token's lookups, of which a thread has 4 on their way: 1000003 tokens of
// 500 requests 12.8 us with cold caches, about what the host takes for the call.
// Whether a batch fits comes from the same sums, in the first block.
#include <cuda_runtime.h>

#include "lik_internal.h"
#include "serve.h"

namespace lik {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int64_t kTop = INT32_MAX;

__device__ __forceinline__ int clamp_top(int64_t v) { return static_cast<int>(v < kTop ? v : kTop); }

struct Request {
    int64_t cached, added, held, need;
};

__device__ __forceinline__ Request request_of(const SlotsArgs& a, int b) {
    Request r;
    const int c = a.cached[b], n = a.added[b], h = a.held[b];
    r.cached = c > 0 ? c : 0;
    r.added = n > 0 ? n : 0;
    r.held = h < 0 ? 0 : (h < a.cols ? h : a.cols);
    const int64_t page = int64_t(1) << a.page_shift;
    int64_t want = (r.cached + r.added + page - 1) >> a.page_shift;
    want = want < a.cols ? want : a.cols;
    r.need = want > r.held ? want - r.held : 0;
    return r;
}

// The last index i in [0, n) with prefix[i] <= t; prefix[0] = 0 <= t.
__device__ __forceinline__ int find(const int* prefix, int n, int t) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (prefix[mid] <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kThreads) cache_slots_kernel(const SlotsArgs a) {
    // new tokens and new pages before a request [requests + 1], both held under 2^31; what it had [requests]
    extern __shared__ int prefix[];
    int* const tokens = prefix;
    int* const pages = tokens + a.requests + 1;
    int* const had = pages + a.requests + 1;
    int* const held = had + a.requests;
    __shared__ int64_t warp_tokens[kWarps], warp_pages[kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = a.requests;

    // a thread sums neighbouring requests, then warps and block join the sums
    const int each = (B + kThreads - 1) / kThreads;
    const int b0 = min(tid * each, B), b1 = min(b0 + each, B);
    int64_t st = 0, sp = 0;
    for (int b = b0; b < b1; ++b) {
        const Request r = request_of(a, b);
        st += r.added;
        sp += r.need;
    }
    int64_t it = st, ip = sp;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const int64_t t = __shfl_up_sync(0xffffffffu, it, d), p = __shfl_up_sync(0xffffffffu, ip, d);
        if (lane >= d) {
            it += t;
            ip += p;
        }
    }
    if (lane == 31) {
        warp_tokens[warp] = it;
        warp_pages[warp] = ip;
    }
    __syncthreads();
    int64_t all_tokens = 0, all_pages = 0;
    it -= st;
    ip -= sp;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) {
            it += warp_tokens[w];
            ip += warp_pages[w];
        }
        all_tokens += warp_tokens[w];
        all_pages += warp_pages[w];
    }
    int64_t count = *a.free_count;
    count = count < 0 ? 0 : (count < a.free_capacity ? count : a.free_capacity);
    const bool first = blockIdx.x == 0;
    int64_t lost = 0;  // new tokens without a row or a page
    for (int b = b0; b < b1; ++b) {
        const Request r = request_of(a, b);
        tokens[b] = clamp_top(it);
        pages[b] = clamp_top(ip);
        had[b] = static_cast<int>(r.cached);
        held[b] = static_cast<int>(r.held);
        if (first) {
            const int64_t left = count - ip;
            const int64_t got = left <= 0 ? 0 : (r.need < left ? r.need : left);
            a.held_out[b] = static_cast<int>(r.held + got);
            const int64_t row0 = it < a.capacity ? it : a.capacity;
            a.offsets[b] = clamp_top(row0);
            int64_t kept = r.added;
            if (a.missing) {
                const int64_t row1 = it + r.added < a.capacity ? it + r.added : a.capacity;
                kept = row1 - row0;
                const int64_t room = ((r.held + got) << a.page_shift) - r.cached;
                const int64_t placed = kept < room ? kept : room;
                lost += r.added - (placed > 0 ? placed : 0);
            }
            a.lengths[b] = clamp_top(r.cached + kept);
        }
        it += r.added;
        ip += r.need;
    }
    const int n_tokens = clamp_top(all_tokens < a.capacity ? all_tokens : a.capacity);
    const int n_pages = clamp_top(all_pages);
    if (tid == 0) {
        tokens[B] = clamp_top(all_tokens);
        pages[B] = n_pages;
        if (first) {
            a.offsets[B] = n_tokens;
            const int64_t left = count - all_pages;
            *a.free_left = static_cast<int>(left > -kTop ? left : -kTop);
        }
    }
    __syncthreads();
    if (first && a.missing) {  // the block's sums of tokens are no longer needed
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) lost += __shfl_xor_sync(0xffffffffu, lost, d);
        if (lane == 0) warp_tokens[warp] = lost;
        __syncthreads();
        int64_t missing = all_pages - count, pages_lost = 0;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) pages_lost += warp_tokens[w];
        pages_lost = (pages_lost + (int64_t(1) << a.page_shift) - 1) >> a.page_shift;
        missing = missing > pages_lost ? missing : pages_lost;
        if (tid == 0) *a.missing = clamp_top(missing);
        for (int b = b0; b < b1; ++b) a.most[b] = missing ? had[b] : a.lengths[b];  // its own writes
    }

    const int64_t step = static_cast<int64_t>(gridDim.x) * kThreads;
    // slots; a token's page is one that its request held, or one of this call's,
    // taken from the list itself: no block reads what another writes
    // A warp takes 32 * kTurn tokens, of which most are a prompt's: the request before is looked at first.
    constexpr int kTurn = 4;
    const int cols = static_cast<int>(a.cols);
    for (int64_t t0 = (blockIdx.x * static_cast<int64_t>(kThreads) + (tid & ~31)) * kTurn + lane; t0 < a.capacity;
         t0 += kTurn * step) {
        const int32_t* from[kTurn];
        uint32_t inside[kTurn];
        int32_t page[kTurn];
        int b = -1;
#pragma unroll
        for (int u = 0; u < kTurn; ++u) {
            from[u] = nullptr;
            inside[u] = 0;
            if (t0 + 32 * u < n_tokens) {
                const int t = static_cast<int>(t0) + 32 * u;
                if (b < 0 || tokens[b + 1] <= t) b = find(tokens, B, t);
                const uint32_t pos = static_cast<uint32_t>(had[b]) + static_cast<uint32_t>(t - tokens[b]);
                const int col = static_cast<int>(pos >> a.page_shift), own = held[b];
                inside[u] = pos & ((1u << a.page_shift) - 1);
                if (col < own) {
                    from[u] = a.table + b * a.stride + col;
                } else if (col < cols) {
                    const int64_t at = count - 1 - pages[b] - (col - own);
                    if (at >= 0) from[u] = a.free_pages + at;
                }
            }
        }
#pragma unroll
        for (int u = 0; u < kTurn; ++u) page[u] = from[u] ? *from[u] : -1;
#pragma unroll
        for (int u = 0; u < kTurn; ++u)
            if (t0 + 32 * u < a.capacity)
                a.slots[t0 + 32 * u] = page[u] >= 0 ? (static_cast<int64_t>(page[u]) << a.page_shift) + inside[u] : -1;
    }
    for (int64_t r = blockIdx.x * static_cast<int64_t>(kThreads) + tid; r < n_pages; r += step) {
        const int ri = static_cast<int>(r);
        const int q = find(pages, B, ri);
        const int64_t at = count - 1 - r;
        a.table[q * a.stride + held[q] + (ri - pages[q])] = at >= 0 ? a.free_pages[at] : -1;
    }
}

}  // namespace

cudaError_t launch_cache_slots(const SlotsArgs& a, cudaStream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const int64_t work = a.capacity > a.requests ? a.capacity : a.requests;
    const int64_t most = 2 * device_info(dev).sm_count;
    int64_t blocks = (work + 4 * kThreads - 1) / (4 * kThreads);
    blocks = blocks < 1 ? 1 : (blocks < most ? blocks : most);
    const size_t smem = sizeof(int) * (4 * static_cast<size_t>(a.requests) + 2);
    if (smem > 48 * 1024) {
        e = cudaFuncSetAttribute(cache_slots_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 sizeof(int) * (4 * kMaxRequests + 2));
        if (e != cudaSuccess) return e;
    }
    cache_slots_kernel<<<static_cast<unsigned>(blocks), kThreads, smem, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace lik
