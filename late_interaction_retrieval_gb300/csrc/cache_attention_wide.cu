// cache_attention_wide.cu -- attention over the 8-bit cache for many rows a
// key head (drafts of grouped heads, prompts): the products on tcgen05.
//
// A tile is 64 tokens against 128 rows: S = Q K^T in tensor memory, its
// softmax weights back into tensor memory as fp16, O += P V.  There are two
// streams with a softmax warpgroup, two S/P and an O accumulator each, so that
// the tensor cores work on one while the other's exponentials are taken.
// Where an item has more than 128 rows the streams are its two halves, on the
// same tokens (the codes are widened once for both); else they are the even
// and the odd tiles of the same rows, joined at the item's end.
//
// The codes become fp16 (exactly) on their way from the TMA ring to the MMA's
// operand tiles.  K stays token by token.  V is transposed, so that both
// operands are K-major: a thread takes 8 tokens of 8 dimensions, byte
// permutes pair the tokens, and every store is 16 bytes.  Those 8 tokens lie
// 8 apart in a block of 64 (which keeps the loads free of bank conflicts), so
// the tokens of S's columns are ordered that way: column j of a block holds
// token (j mod 8) * 8 + j / 8.
//
// The weights are 2^7 exp2(z - ref) (the page's scale / c) in fp16.  ref is a
// power of two near the row's largest weight and c one not below the scales;
// either moves only when a weight leaves fp16's range, which its sum shows (no
// maximum is taken on the way), and its move rescales O, exactly.  For fp16
// outputs, where 11 bits of a weight would show, what their rounding left is
// multiplied too, from the columns of S that the weights leave free.  Work is
// spread by costs in closed form, the batch's items end to end, one equal
// range a block; pieces of cut items are joined by a second launch.
//
// What bounds it: neither memory nor the tensor cores (41% busy) but the chain
// weights -> O and next scores -> weights of a stream (2000 clocks a tile, of
// which the tensor cores take 620), 14000 clocks at an item's start and end,
// and with one stream's rows the widening of the codes.  8191 new tokens over
// 16381, 32 heads, bf16: 480 to 530 us, 780 to 860 TFLOP/s; fp16 with its second
// product 630 to 720 us; 48 requests of 5 drafts over 150001 tokens, 64 heads,
// fp16: 178 us.
#include "cache_attention.h"
#include "tmap.h"

namespace lik {
namespace {

using namespace attn;

constexpr int kThreads = 640;
constexpr int kTok = 64;
constexpr int kM = 128;
constexpr int kItemRows = 256;
constexpr int kRaw = 6;         // raw tiles of one operand
constexpr int kKeys = 3, kValues = 4;  // operand tiles
constexpr int kAhead = 2;       // steps of a stream whose scores are computed ahead
constexpr int kScaleRing = 16;  // tiles whose scales are kept
// warps
constexpr int kConvert = 8, kLoad = 16, kMma = 17, kBusy = 19;  // converters of K, of V; an issuer of MMAs a stream

constexpr float kHalfMost = 65504.0f;  // the largest finite fp16
constexpr float kLogLimit = 9.5f;      // 64 weights of 2^9.5 are below it together

constexpr uint32_t kColS = 0, kColO = 256;

struct PieceInfo {
    int request, head, item;  // request -1: no piece
    int begins, ends;
};

template <int DP>
struct Smem {
    alignas(1024) uint8_t q[2][DP / 64][kM * 128];
    uint8_t k[kKeys][DP / 64][kTok * 128];
    uint8_t v[kValues][DP * 128];
    uint8_t raw[kRaw][kTok * DP];
    float4 scale[kScaleRing][4];  // of 16 tokens each: keys', values', log2 of the latter
    uint32_t valid[kScaleRing];
    uint64_t raw_full[kRaw], raw_empty[kRaw], scale_full[kScaleRing];
    uint64_t k_full[kKeys], k_empty[kKeys], v_full[kValues], v_empty[kValues];
    uint64_t q_full[2], s_full[2][2], p_full[2][2];
    uint64_t o_most[2], o_full[2];  // all of an item's steps but the last are in O; all are
    uint64_t merge_full, merge_empty, exit_bar;
    uint32_t tmem;
    int nan_seen;
    int start[4], end[4];  // request, head, item, tile
    long long warp_sum[kThreads / 32];
};

struct Maps {
    CUtensorMap k, v;
};

// 256 rows (or what is left) of a request's (token, query head of the key head).
struct Item {
    Request r;
    int b, head, item;
    int rows;   // of the item
    int tiles;  // of 128 tokens that any of its rows sees, at least 1
    bool two;   // more than 128 rows: a stream for each half
};

__device__ __forceinline__ int items_of(const Request& r, int group) { return (r.n * group + kItemRows - 1) / kItemRows; }

__device__ __forceinline__ void shape(Item& x, int group) {
    const int all = x.r.n * group, first = x.item * kItemRows;
    x.rows = min(kItemRows, all - first);
    x.two = x.rows > kM;
    const int sees = min(x.r.before + (first + x.rows - 1) / group + 1, x.r.length);
    x.tiles = max(1, (sees + kTok - 1) / kTok);
}

// What items cost, in closed form, so that a block finds its range without a walk over the batch.  The unit is a token
// of one stream and one row group of a stream's 128: an item of both streams costs 2 group (tokens that its last row
// sees + kItemCost), 256 rows being 256 / group tokens, which is counted group times and so stays whole; one of a
// single stream's rows, whose tiles the streams share, half of that and as much again for its start and end.
constexpr int kItemCost = 416;  // tokens: q, the output, and the rest of the last tile (14000 clocks, a tile 2000)

struct Costs {
    long long each, last;  // 2 group (tokens before the request's new ones + kItemCost); the last item's
    int items;
    // of the items before item i
    __device__ __forceinline__ long long before(int i) const { return i * each + static_cast<long long>(kItemRows) * i * (i + 1); }
    __device__ __forceinline__ long long all() const { return before(items - 1) + last; }  // of a key head
};

__device__ __forceinline__ Costs costs_of(const Request& r, int group) {
    Costs c;
    c.items = items_of(r, group);
    const long long base = max(r.length - r.n, 0);
    const int rows = r.n * group - (c.items - 1) * kItemRows;
    c.each = 2 * group * (base + kItemCost);
    c.last = rows > kM ? c.each + 2ll * r.n * group : group * (base + 2 * kItemCost) + r.n * group;
    return c;
}

// Walks a block's segments: an item and a range of its tiles.  The range's end
// stays in shared memory.
struct Walk {
    Item x;
    int t0, t1;
    bool last;
    const int* end;
    __device__ __forceinline__ void place(int group, int tile) {
        shape(x, group);
        last = x.b == end[0] && x.head == end[1] && x.item == end[2];
        t0 = tile;
        t1 = last ? end[3] : x.tiles;
    }
    __device__ __forceinline__ void begin(const AttentionArgs& a, int group, const int* from, const int* to) {
        end = to;
        x.b = from[0];
        x.head = from[1];
        x.item = from[2];
        x.r = request_of(a, x.b);
        place(group, from[3]);
    }
    __device__ __forceinline__ void next(const AttentionArgs& a, int group) {
        if (++x.item >= items_of(x.r, group)) {
            x.item = 0;
            if (++x.head >= a.heads) {
                x.head = 0;
                do {
                    x.r = request_of(a, ++x.b);
                } while (x.r.n == 0);  // the end's request has rows
            }
        }
        place(group, 0);
    }
};

__device__ __forceinline__ uint4 lds16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
    return v;
}
__device__ __forceinline__ uint2 lds8(uint32_t at) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(at));
    return v;
}
__device__ __forceinline__ uint32_t lds4(uint32_t at) {
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(at));
    return v;
}
__device__ __forceinline__ void sts8(uint32_t at, uint32_t x, uint32_t y) {
    asm volatile("st.shared.v2.u32 [%0], {%1, %2};" ::"r"(at), "r"(x), "r"(y) : "memory");
}
__device__ __forceinline__ void sts16(uint32_t at, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
// Shared memory written by this thread, before the tensor cores read it.
__device__ __forceinline__ void fence_operands() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 16-byte chunk c of row r of a raw tile as TMA swizzles it.
template <int DP>
__device__ __forceinline__ uint32_t raw_at(int r, int c) {
    return DP == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}
// 16-byte chunk c of row r of an operand tile with rows of 128 bytes, swizzled.
__device__ __forceinline__ uint32_t tile_at(int r, int c) { return r * 128 + ((c ^ (r & 7)) << 4); }

// D (+)= A B^T with A (fp16, two to a 32-bit column) in tensor memory.
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u)
        : "memory");
}

__device__ __forceinline__ void tmem_st_16(uint32_t taddr, const uint32_t (&v)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
        "%12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
        : "memory");
}

// 32 columns of this thread's lane, on their way: fence_loaded() before they are used.
__device__ __forceinline__ void tmem_ld_32(uint32_t taddr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(taddr)
        : "memory");
}
// Waits for the loads; every use of v comes behind it.
__device__ __forceinline__ void fence_loaded(uint32_t (&v)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                   "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                   "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]),
                   "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                   "+r"(v[30]), "+r"(v[31])
                 :
                 : "memory");
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
__device__ __forceinline__ uint64_t fma_both(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t add_both(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}

// The larger of either half's 16 bits.
__device__ __forceinline__ uint32_t max_halves(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.u16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}

// One thread of the warp.
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

// Registers of a warpgroup's threads: 256 threads of 144 and 384 of 64 are the
// 640 of 96 that the block is launched with.
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 144;"); }
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 64;"); }

__device__ __forceinline__ uint32_t pack_out(float x, float y, bool bf16) {
    if (!bf16) return pack_half(x, y);
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// N neighbouring dimensions of one row to the output; wide: the bytes that its rows are aligned to (32: a sector in
// one store).
template <int N>
__device__ __forceinline__ void store(void* out, int64_t at, const float (&f)[N], bool bf16, int wide) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) w[i] = pack_out(f[2 * i], f[2 * i + 1], bf16);
    uint16_t* const p = static_cast<uint16_t*>(out) + at;
    if (N == 16 && wide >= 32) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[N / 2 - 4]), "r"(w[N / 2 - 3]), "r"(w[N / 2 - 2]), "r"(w[N / 2 - 1])
                     : "memory");
    } else if (wide >= 16) {
#pragma unroll
        for (int i = 0; i < N / 8; ++i)
            reinterpret_cast<uint4*>(p)[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    } else {
#pragma unroll
        for (int i = 0; i < N / 2; ++i) {
            p[2 * i] = static_cast<uint16_t>(w[i]);
            p[2 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
        }
    }
}

template <int DP, bool kFine>
__global__ void __launch_bounds__(kThreads, 1)
    attention_wide_kernel(const AttentionArgs a, const __grid_constant__ Maps maps, unsigned int* err,
                          PieceInfo* infos, float* pieces, int piece_rows, bool q_wide, int out_wide) {
    extern __shared__ uint8_t raw_smem[];
    Smem<DP>& sm = *reinterpret_cast<Smem<DP>*>((reinterpret_cast<uintptr_t>(raw_smem) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = a.q_heads / a.heads;
    const bool bf16 = a.dtype == kBF16;
    using ptx::smem_u32;

    if (tid == 0) {
        for (int i = 0; i < kRaw; ++i) {
            ptx::mbar_init(smem_u32(&sm.raw_full[i]), 1);
            ptx::mbar_init(smem_u32(&sm.raw_empty[i]), 4);
        }
        for (int i = 0; i < kScaleRing; ++i) ptx::mbar_init(smem_u32(&sm.scale_full[i]), 1);
        for (int i = 0; i < kKeys; ++i) {
            ptx::mbar_init(smem_u32(&sm.k_full[i]), 4);
            ptx::mbar_init(smem_u32(&sm.k_empty[i]), 2);
        }
        for (int i = 0; i < kValues; ++i) {
            ptx::mbar_init(smem_u32(&sm.v_full[i]), 4);
            ptx::mbar_init(smem_u32(&sm.v_empty[i]), 2);
        }
        for (int i = 0; i < 2; ++i) {
            ptx::mbar_init(smem_u32(&sm.q_full[i]), 4);
            ptx::mbar_init(smem_u32(&sm.o_most[i]), 1);
            ptx::mbar_init(smem_u32(&sm.o_full[i]), 1);
            for (int b = 0; b < 2; ++b) {
                ptx::mbar_init(smem_u32(&sm.s_full[i][b]), 1);
                ptx::mbar_init(smem_u32(&sm.p_full[i][b]), 4);
            }
        }
        ptx::mbar_init(smem_u32(&sm.merge_full), 4);
        ptx::mbar_init(smem_u32(&sm.merge_empty), 4);
        ptx::mbar_init(smem_u32(&sm.exit_bar), kBusy);
        sm.nan_seen = 0;
        ptx::fence_mbar_init();
    }
    // ---- the block's range of the batch, by costs, from every request's
    // Either half of the block sums all requests, and finds one of the range's bounds.
    constexpr int kHalf = kThreads / 2;
    const int half = tid >= kHalf, part = tid - half * kHalf;
    const int B = a.requests, each = (B + kHalf - 1) / kHalf;
    auto cost_of = [&](int b) {
        const Request r = request_of(a, b);
        return r.n > 0 ? costs_of(r, group).all() * a.heads : 0ll;
    };
    long long mine = 0;
    for (int b = min(part * each, B); b < min(part * each + each, B); ++b) mine += cost_of(b);
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) sm.warp_sum[warp] = incl;
    __syncthreads();
    long long all = 0;
    for (int w = half * (kHalf / 32); w < (half + 1) * (kHalf / 32); ++w) {
        if (w < warp) incl += sm.warp_sum[w];
        all += sm.warp_sum[w];
    }
    const long long excl = incl - mine;
    if (tid < 2) infos[2 * blockIdx.x + tid] = PieceInfo{-1, 0, 0, 0, 0};
    // a block has two steps (a tile of one stream) at least, or thereabouts
    const long long active = max(1ll, min(static_cast<long long>(gridDim.x), all / (2 * kTok * group)));
    if (all == 0 || blockIdx.x >= active) return;
    auto bound = [&](long long k) { return all / active * k + all % active * k / active; };
    // the tile that a cost u falls on, by the thread whose requests do; the batch's end comes behind its last tile
    auto locate = [&](long long u, int* to) {
        const bool behind = u == all;
        u -= behind;
        if (u < excl || u >= incl) return;
        long long rest = u - excl;
        int b = part * each;
        for (long long c = cost_of(b); rest >= c; c = cost_of(++b)) rest -= c;
        const Request r = request_of(a, b);
        const Costs c = costs_of(r, group);
        to[0] = b;
        const long long per_head = c.all();
        to[1] = static_cast<int>(rest / per_head);
        rest -= to[1] * per_head;
        int i = 0;  // the last item that begins at or before it
        for (int step = 1 << (31 - __clz(c.items)); step; step >>= 1)
            if (i + step < c.items && c.before(i + step) <= rest) i += step;
        Item x;
        x.r = r;
        x.item = i;
        shape(x, group);
        // the same rounding for the block that ends here and the one that begins
        const float cost = static_cast<float>(i + 1 < c.items ? c.before(i + 1) - c.before(i) : c.last);
        to[2] = i;
        to[3] = behind ? x.tiles : min(x.tiles - 1, static_cast<int>(static_cast<float>(rest - c.before(i)) / cost * x.tiles));
    };
    locate(bound(blockIdx.x + half), half ? sm.end : sm.start);
    __syncthreads();
    if (sm.start[0] == sm.end[0] && sm.start[1] == sm.end[1] && sm.start[2] == sm.end[2] && sm.start[3] == sm.end[3])
        return;  // both bounds fall on one tile
    if (warp == kMma) {
        ptx::tmem_alloc(smem_u32(&sm.tmem), 512);
        ptx::tmem_relinquish();
        ptx::tc_fence_before();
    }
    __syncthreads();
    ptx::tc_fence_after();
    const uint32_t tmem = sm.tmem;
    if (warp >= kBusy) {
        fewer_registers();
        return;
    }

    bool ok = true;
    const int page_size = 1 << a.page_shift;

    if (warp == kLoad) {
        // ------------------------------------------------------- raw tiles --
        fewer_registers();
        Walk w;
        w.begin(a, group, sm.start, sm.end);
        const int box = min(page_size, 64);
        int slot = 0;
        uint32_t phase = 1;  // an empty ring
        int n = 0;           // tiles so far
        // a lane looks up 16 tokens of the next 8 tiles, while the 8 before are on their way
        int page = -1;
        float2 scale = make_float2(0.0f, 0.0f);
        auto look_up = [&](int t, int& pg, float2& sc) {
            const int pos = (t + (lane >> 2)) * kTok + 16 * (lane & 3);
            int p = -1;
            if (t + (lane >> 2) < w.t1 && pos < w.x.r.length) p = a.table[w.x.b * a.stride + (pos >> a.page_shift)];
            pg = p >= 0 && p < a.pages ? p : -1;
            sc = make_float2(0.0f, 0.0f);
            if (pg >= 0) {
                sc.x = a.k_scale[static_cast<int64_t>(pg) * a.heads + w.x.head];
                sc.y = a.v_scale[static_cast<int64_t>(pg) * a.heads + w.x.head];
            }
        };
        while (ok) {
            int next_page;
            float2 next_scale;
            look_up(w.t0, next_page, next_scale);
            for (int t = w.t0; ok && t < w.t1; ++t, ++n) {
                const int of = (t - w.t0) & 7;  // of the lanes' tiles
                if (of == 0) {
                    page = next_page;
                    scale = next_scale;
                    look_up(t + 8, next_page, next_scale);
                }
                const int now = __shfl_sync(0xffffffffu, page, 4 * of + (lane & 3));
                const uint32_t live = __ballot_sync(0xffffffffu, lane < 4 && now >= 0);
                const int at = n & (kScaleRing - 1);
                if (lane >> 2 == of)
                    sm.scale[at][lane & 3] = make_float4(scale.x, scale.y, __log2f(scale.y), 0.0f);
                if (lane == 0) sm.valid[at] = live;
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(smem_u32(&sm.scale_full[at]));
#pragma unroll 1
                for (int part = 0; part < 2; ++part) {  // keys, values
                    ok = __all_sync(0xffffffffu, ptx::mbar_wait(smem_u32(&sm.raw_empty[slot]), phase, err));
                    if (!ok) break;
                    const uint32_t bar = smem_u32(&sm.raw_full[slot]);
                    if (lane == 0) {
                        if (live) ptx::mbar_arrive_expect_tx(bar, kTok * DP);
                        else ptx::mbar_arrive(bar);  // nothing to load
                    }
                    __syncwarp();
                    // a lane loads what begins at its 16 tokens
                    if (live && lane < 4 && 16 * lane % box == 0) {
                        const int off = w.x.head * page_size + ((t * kTok + 16 * lane) & (page_size - 1));
                        ptx::tma_load_3d(smem_u32(&sm.raw[slot][16 * lane * DP]), part ? &maps.v : &maps.k, 0, off,
                                         max(now, 0), bar);
                    }
                    if (++slot == kRaw) {
                        slot = 0;
                        phase ^= 1;
                    }
                }
            }
            if (!ok || w.last) break;
            w.next(a, group);
        }
    } else if (warp >= kConvert && warp < kConvert + 8) {
        // ----------------------------------------------- codes to operands --
        fewer_registers();
        Walk w;
        w.begin(a, group, sm.start, sm.end);
        const int ct = tid & 127;
        const bool keys = warp < kConvert + 4;
        int n = 0, slot = keys ? 0 : 1, buf = 0;
        uint32_t raw_phase = 0, phase = 1;  // full raw tiles, empty operand tiles
        const int buffers = keys ? kKeys : kValues;
        uint64_t* const empty = keys ? sm.k_empty : sm.v_empty;
        while (ok) {
            // what even the item's first row sees
            const int all_see = w.x.r.before + (w.x.item * kItemRows) / group + 1;
#pragma unroll 1
            for (int t = w.t0; t < w.t1; ++t, ++n) {
                ok = ptx::mbar_wait(smem_u32(&empty[buf]), phase, err) &&
                     ptx::mbar_wait(smem_u32(&sm.raw_full[slot]), raw_phase, err);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const uint32_t src = smem_u32(sm.raw[slot]);
                if (keys) {
                    // a thread widens 16 dimensions of a token at a time
                    const uint32_t dst = smem_u32(sm.k[buf][0]);
                    constexpr int C = DP / 16;  // chunks of a token
#pragma unroll 4
                    for (int i = 0; i < kTok * C / 128; ++i) {
                        const int item = ct + 128 * i, c = item % C, tok = item / C;
                        const uint4 x = lds16(src + raw_at<DP>(tok, c));
                        const int row = (tok & 7) * 8 + (tok >> 3);
                        const uint32_t at = dst + (c >> 2) * (kTok * 128);
                        const uint32_t lo = at + tile_at(row, (c & 3) * 2), hi = at + tile_at(row, (c & 3) * 2 + 1);
                        const uint32_t l0 = widen_low(x.x), l1 = widen_high(x.x), l2 = widen_low(x.y), l3 = widen_high(x.y);
                        const uint32_t h0 = widen_low(x.z), h1 = widen_high(x.z), h2 = widen_low(x.w), h3 = widen_high(x.w);
                        // the two 64-dimension tiles share their banks: their lanes take turns
                        if (c & 4) {
                            sts16(hi, h0, h1, h2, h3);
                            sts16(lo, l0, l1, l2, l3);
                        } else {
                            sts16(lo, l0, l1, l2, l3);
                            sts16(hi, h0, h1, h2, h3);
                        }
                    }
                } else {
                    // 8 tokens, 8 apart, of 8 dimensions, transposed
                    const uint32_t dst = smem_u32(sm.v[buf]);
                    const uint32_t valid = sm.valid[n & (kScaleRing - 1)];
                    const int first = t * kTok;
                    const int c8 = ct & 7, d8 = ct >> 3;  // tokens 8 i + c8; dimensions 8 d8 ..
                    if (first + kTok > all_see || valid != 15u) {
                        // tokens that no row sees count as 0; of those that only some rows see, NaN codes are set
                        // apart.  A thread mends the codes that it will read.
                        bool nan = false;
#pragma unroll 1
                        for (int i = 0; d8 < DP / 8 && i < 8; ++i) {
                            const int tok = 8 * i + c8, pos = first + tok;
                            const uint32_t at = src + raw_at<DP>(tok, d8 >> 1) + (d8 & 1) * 8;
                            const uint2 x = lds8(at);
                            const bool live = pos < w.x.r.length && ((valid >> (tok >> 4)) & 1u);
                            const uint32_t some = pos >= all_see ? 0xffffffffu : 0u;
                            const uint32_t nx = __vcmpeq4(x.x & 0x7f7f7f7fu, 0x7f7f7f7fu) & some;
                            const uint32_t ny = __vcmpeq4(x.y & 0x7f7f7f7fu, 0x7f7f7f7fu) & some;
                            nan = nan || (live && (nx | ny));
                            sts8(at, live ? x.x & ~nx : 0u, live ? x.y & ~ny : 0u);
                        }
                        if (nan) sm.nan_seen = 1;
                    }
#pragma unroll 1
                    for (int h = 0; d8 < DP / 8 && h < 2; ++h) {
                        uint32_t x[8], p[4][4];  // [dimension][pair of tokens]
#pragma unroll
                        for (int i = 0; i < 8; ++i) x[i] = lds4(src + raw_at<DP>(8 * i + c8, d8 >> 1) + (d8 & 1) * 8 + 4 * h);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t a01 = __byte_perm(x[2 * i], x[2 * i + 1], 0x5140);
                            const uint32_t a23 = __byte_perm(x[2 * i], x[2 * i + 1], 0x7362);
                            p[0][i] = widen_low(a01);
                            p[1][i] = widen_high(a01);
                            p[2][i] = widen_low(a23);
                            p[3][i] = widen_high(a23);
                        }
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            sts16(dst + tile_at(8 * d8 + 4 * h + j, c8), p[j][0], p[j][1], p[j][2], p[j][3]);
                    }
                }
                fence_operands();
                if (keys) {  // the tile's scales too are there before its scores
                    ok = __all_sync(0xffffffffu, ptx::mbar_wait(smem_u32(&sm.scale_full[n & (kScaleRing - 1)]),
                                                                (n / kScaleRing) & 1, err));
                    if (!ok) break;
                }
                __syncwarp();
                if (lane == 0) {
                    ptx::mbar_arrive(smem_u32(&sm.raw_empty[slot]));
                    ptx::mbar_arrive(smem_u32(keys ? &sm.k_full[buf] : &sm.v_full[buf]));
                }
                if ((slot += 2) >= kRaw) {
                    slot -= kRaw;
                    raw_phase ^= 1;
                }
                if (++buf == buffers) {
                    buf = 0;
                    phase ^= 1;
                }
            }
            if (!ok || w.last) break;
            w.next(a, group);
        }
    } else if (warp >= kMma) {
        // ------------------------------------------------------------ MMAs --
        fewer_registers();
        Walk w;
        w.begin(a, group, sm.start, sm.end);
        // The warp goes through it together, one thread of it issues: so the operands are uniform, and an instruction is
        // issued in a third of the clocks that it takes in a branch of one lane.
        constexpr uint32_t kIdS = ptx::f16_idesc(kM, kTok, false), kIdO = ptx::f16_idesc(kM, DP, false);
        const bool leader = elect();
        const int s = warp - kMma;
        const uint32_t col_s = tmem + kColS + 128 * s, col_o = tmem + kColO + 128 * s;
        // descriptors count addresses in 16 bytes
        const uint64_t q0 = ptx::sw128_kmajor_desc(smem_u32(sm.q[s][0])), k0 = ptx::sw128_kmajor_desc(smem_u32(sm.k[0][0])),
                       v0 = ptx::sw128_kmajor_desc(smem_u32(sm.v[0]));
        int n = 0;        // tiles before this segment
        uint32_t sb = 0;  // the buffer of the next scores
        uint32_t ob = 0, p_phase = 0, q_phase = 0;
        auto wait = [&](uint64_t& bar, uint32_t phase) {
            ok = ok && __all_sync(0xffffffffu, ptx::mbar_wait(smem_u32(&bar), phase, err));
        };
        while (ok) {
            const bool two = w.x.two;
            const int tiles = w.t1 - w.t0, steps = two ? tiles : (tiles + 1 - s) / 2;
            // A buffer is empty again when both streams have done with it; a tile of one stream counts twice.
            auto done = [&](uint64_t* bar) {
                ptx::mma_commit(smem_u32(bar));
                if (!two) ptx::mma_commit(smem_u32(bar));
            };
            // This stream's tiles: all of the segment's, or every second one.  Tiles are filled in order, so the other
            // stream's phase between two of this stream's in one buffer has been completed when this one asks for the
            // second.
            const int first = n + (two ? 0 : s), by = two ? 1 : 2;
            int kb = first % kKeys, vb = first % kValues;
            uint32_t k_phase = (first / kKeys) & 1, v_phase = (first / kValues) & 1;
            // The scores of the next tile.  The weights of two steps ago in their place were multiplied by an
            // instruction before these.
            auto score = [&]() {
                wait(sm.k_full[kb], k_phase);
                if (!ok) return;
                ptx::tc_fence_after();
                const uint64_t kd = k0 + kb * (DP / 64 * kTok * 128 / 16);
                const uint32_t d = col_s + 64 * sb;
                if (leader) {
#pragma unroll
                    for (int k = 0; k < DP / 16; ++k)  // 64 dimensions a swizzle atom: 4 steps of 32 bytes
                        ptx::mma_f16(d, q0 + (k >> 2) * (kM * 128 / 16) + 2 * (k & 3),
                                     kd + (k >> 2) * (kTok * 128 / 16) + 2 * (k & 3), kIdS, k != 0);
                    ptx::mma_commit(smem_u32(&sm.s_full[s][sb]));
                    done(&sm.k_empty[kb]);
                }
                sb ^= 1;
                if ((kb += by) >= kKeys) {
                    kb -= kKeys;
                    k_phase ^= 1;
                }
            };
            if (steps > 0) {
                wait(sm.q_full[s], q_phase);
                q_phase ^= 1;
            }
            for (int i = 0; ok && i < min(kAhead, steps); ++i) score();
            for (int i = 0; ok && i < steps; ++i) {
                wait(sm.v_full[vb], v_phase);
                wait(sm.p_full[s][ob], p_phase);
                if (!ok) break;
                ptx::tc_fence_after();
                const uint64_t vd = v0 + vb * (DP * 128 / 16);
                if (leader) {
#pragma unroll
                    for (int k = 0; k < kTok / 16; ++k)
                        mma_f16_ts(col_o, col_s + 64 * ob + 8 * k, vd + 2 * k, kIdO, i > 0 || k != 0);
#pragma unroll
                    for (int k = 0; kFine && k < kTok / 16; ++k)
                        mma_f16_ts(col_o, col_s + 64 * ob + 32 + 8 * k, vd + 2 * k, kIdO, true);
                }
                // the next scores first: the softmax waits for them
                if (i + kAhead < steps) score();
                if (leader) {
                    if (i + 2 == steps) ptx::mma_commit(smem_u32(&sm.o_most[s]));
                    if (i + 1 == steps) ptx::mma_commit(smem_u32(&sm.o_full[s]));
                    done(&sm.v_empty[vb]);
                }
                p_phase ^= ob;
                ob ^= 1;
                if ((vb += by) >= kValues) {
                    vb -= kValues;
                    v_phase ^= 1;
                }
            }
            n += tiles;
            if (!ok || w.last) break;
            w.next(a, group);
        }
        __syncwarp();
    } else {
        // --------------------------------------------------------- softmax --
        more_registers();
        Walk w;
        w.begin(a, group, sm.start, sm.end);
        const int s = warp >> 2, row = tid & 127;
        const uint32_t lanes = static_cast<uint32_t>(warp & 3) << 21;  // the warp's 32 lanes of tensor memory
        const uint32_t col_o = tmem + lanes + kColO + 128 * s;
        const uint32_t q_tile = smem_u32(sm.q[s][0]);
        auto steps_here = [&](const Walk& x) { return x.x.two ? x.t1 - x.t0 : (x.t1 - x.t0 + 1 - s) / 2; };
        // The warp's rows of x's q on their way into the operand tile, as they are: the lanes of a row's chunks next to
        // one another, so that whole rows are read.
        auto fetch = [&](const Walk& x) {
            if (steps_here(x) <= 0) return false;
            const int in_item = (x.x.two ? s * kM : 0) + row;
            const bool live = in_item < x.x.rows;
            const int rr = live ? x.x.item * kItemRows + in_item : 0;
            const int i = rr / group, h = x.x.head * group + (rr - i * group);
            const uint16_t* const src =
                static_cast<const uint16_t*>(a.q) + (x.x.r.row0 + i) * a.q_token_stride + h * a.q_head_stride;
            if (q_wide) {
                constexpr int C = DP / 8, R = 32 / C;  // chunks of a row, rows at a time
                const int c = lane % C;
                const uint32_t to = q_tile + (c >> 3) * (kM * 128);
#pragma unroll 4
                for (int r = lane / C; r < 32; r += R) {
                    const uint16_t* const from = reinterpret_cast<const uint16_t*>(
                        __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(live ? src : nullptr), r));
                    const uint32_t at = to + tile_at((warp & 3) * 32 + r, c & 7);
                    if (from && c * 8 < a.dim)
                        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(at), "l"(from + c * 8) : "memory");
                    else
                        sts16(at, 0, 0, 0, 0);
                }
            } else {
#pragma unroll 1
                for (int c = 0; c < DP / 8; ++c) {
                    uint32_t e[4] = {0, 0, 0, 0};
                    if (live && c * 8 < a.dim) {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            e[k] = src[8 * c + 2 * k] | (static_cast<uint32_t>(src[8 * c + 2 * k + 1]) << 16);
                    }
                    sts16(q_tile + (c >> 3) * (kM * 128) + tile_at(row, c & 7), e[0], e[1], e[2], e[3]);
                }
            }
            return true;
        };
        // The thread's row, scaled to fp16's range in its place; the factor of its scores.
        auto convert = [&]() {
            asm volatile("cp.async.wait_all;" ::: "memory");
            __syncwarp();
            float2 down = make_float2(1.0f, 1.0f);
            if (bf16) {
                uint32_t sizes = 0;  // the largest size's bits of either half
#pragma unroll 4
                for (int c = 0; c < DP / 8; ++c) {
                    const uint4 e = lds16(q_tile + (c >> 3) * (kM * 128) + tile_at(row, c & 7));
                    sizes = max_halves(max_halves(sizes, e.x & 0x7fff7fffu), e.y & 0x7fff7fffu);
                    sizes = max_halves(max_halves(sizes, e.z & 0x7fff7fffu), e.w & 0x7fff7fffu);
                }
                const int shift = row_shift(widen_q(max(sizes & 0xffffu, sizes >> 16), true).x);
                const float2 up = power_of_two(shift);
                down = power_of_two(-shift);
#pragma unroll 2
                for (int c = 0; c < DP / 8; ++c) {
                    const uint32_t at = q_tile + (c >> 3) * (kM * 128) + tile_at(row, c & 7);
                    const uint4 v = lds16(at);
                    const uint32_t e[4] = {v.x, v.y, v.z, v.w};
                    uint32_t o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float2 f = widen_q(e[j], true);
                        o[j] = pack_half(f.x * up.x * up.y, f.y * up.x * up.y);
                    }
                    sts16(at, o[0], o[1], o[2], o[3]);
                }
            }
            fence_operands();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(smem_u32(&sm.q_full[s]));
            return a.scale * 1.44269504088896341f * down.x * down.y;
        };
        int n = 0, count = 0;  // tiles, and steps of this stream, before
        uint32_t most_phase = 0, o_phase = 0, merge_phase = 0;
        float factor = fetch(w) ? convert() : 0.0f;
        while (ok) {
            const bool two = w.x.two;
            const int tiles = w.t1 - w.t0, steps = steps_here(w);
            const int in_item = (two ? s * kM : 0) + row;
            const bool live = in_item < w.x.rows;
            const int rr = w.x.item * kItemRows + in_item;  // of the request's rows
            const int i = live ? rr / group : 0;
            const int h = w.x.head * group + (live ? rr % group : 0);
            const int sees = live ? w.x.r.before + i + 1 : 0;
            const int all_see = w.x.r.before + (w.x.item * kItemRows) / group + 1;
            const bool idle = __ballot_sync(0xffffffffu, live) == 0;  // no row of this warp's: its weights do not matter
            // have: the row has a reference, from its first token's score, whatever that is; 0 stands in before
            float ref = 0.0f, l = 0.0f, cref = 0.0f, logc = -127.0f;  // logc: log2 of cref
            bool have = false;
            bool nan_scale = false;  // the row sees a page whose values' scale is not finite
            // The next item's q is fetched once this one's last scores are there, and is an operand before this one's
            // output is written.
            bool more = false;  // it has tiles of this stream
            auto fetch_next = [&]() {
                if (w.last) return;
                Walk x = w;
                x.next(a, group);
                more = fetch(x);
            };
            if (steps == 0) fetch_next();
            // O times `keep` (1 in rows that need none) in step st > 0.  It is at rest once the step before is in it:
            // this step's product waits for its weights.  The next step's scores are issued behind the product of the
            // step before, and their commit covers it; they wait for nothing of this step.  An item's last step has none
            // behind it: its barrier is waited for in every item, at the latest at its end.  So either barrier is waited
            // for in each of its phases, and is at most one ahead.
            auto rescale = [&](bool last, float keep) {
                const int next = count + 1;
                const uint32_t bar = smem_u32(last ? &sm.o_most[s] : &sm.s_full[s][next & 1]);
                if (!__all_sync(0xffffffffu, ptx::mbar_wait(bar, last ? most_phase : (next >> 1) & 1, err))) return false;
                ptx::tc_fence_after();
#pragma unroll 1
                for (int c = 0; c < DP / 16; ++c) {
                    uint32_t o[16];
                    ptx::tmem_ld_16(col_o + 16 * c, o);
#pragma unroll
                    for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * keep);
                    tmem_st_16(col_o + 16 * c, o);
                }
                return true;
            };
#pragma unroll 1
            for (int st = 0; st < steps; ++st) {
                const int t = two ? st : 2 * st + s;  // of the segment
                const int at = (n + t) & (kScaleRing - 1), tok0 = (w.t0 + t) * kTok;
                const int b = count & 1;
                const uint32_t col_s = tmem + lanes + kColS + 128 * s + 64 * b;
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(smem_u32(&sm.s_full[s][b]), (count >> 1) & 1, err));
                if (!ok) break;
                ptx::tc_fence_after();
                if (st + 1 == steps) fetch_next();
                if (!idle) {
                    const uint32_t valid = sm.valid[at];
                    const bool whole = tok0 + kTok <= all_see && valid == 15u;
                    const bool even = whole && page_size >= 64;  // one page, no token hidden
                    // 16 tokens that share their scales: the columns with (j mod 8) / 2 alike
                    float fk[4], lw[4], minus[4];
                    // log2 of a group's weight (c: 2^7).  2^-60 of c stands in for smaller scales (their fp16
                    // weights are 0 then) and for one that is not finite, which makes the whole row's output NaN: the
                    // sums do not depend on it.  A factor is never 0: a hidden token's score is -inf.  A factor that
                    // is not finite does not reach rows that see none of its tokens.
                    auto weigh = [&](float4 x, bool seen, float& f, float& w) {
                        f = x.x * factor;
                        f = f <= 1e-37f || !seen ? 1e-37f : f;
                        const bool finite = x.y <= 3.402823466e38f;
                        nan_scale = nan_scale || (seen && !finite);
                        w = x.y > cref * 8.67361738e-19f && finite ? x.z + (kLogStart - logc) : kLogStart - 60.0f;
                    };
                    // A tile that every row sees whole, under the reference as it is (the first has none): no maximum is
                    // taken.  A weight beyond fp16's range shows in the sum, and the weights are only stored if there
                    // is none.
                    bool fits = false;
                    if (whole && st > 0) {
                        uint32_t x[32], y[32], p[16], r[16], p_rest[16], r_rest[16];
                        tmem_ld_32(col_s, x);
                        float vmost = 0.0f;
                        if (even) {
                            const float4 sc = sm.scale[at][0];
                            weigh(sc, true, fk[0], lw[0]);
                            vmost = sc.y;
#pragma unroll
                            for (int k = 1; k < 4; ++k) {
                                fk[k] = fk[0];
                                lw[k] = lw[0];
                            }
                        } else {
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const float4 sc = sm.scale[at][k];
                                weigh(sc, true, fk[k], lw[k]);
                                vmost = sc.y <= vmost ? vmost : sc.y;  // a NaN stays
                            }
                        }
                        uint64_t f2[4], m2[4], s2[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            f2[k] = both(fk[k], fk[k]);
                            m2[k] = both(lw[k] - ref, lw[k] - ref);
                            s2[k] = 0;
                        }
                        auto weights = [&](const uint32_t (&v)[32], uint32_t (&to)[16], uint32_t (&rest)[16]) {
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const int k = i & 3;
                                const float2 z = each_of(fma_both(both(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1])),
                                                                  f2[k], m2[k]));
                                const float e0 = exp2_fast(z.x), e1 = exp2_fast(z.y);
                                s2[k] = add_both(s2[k], both(e0, e1));
                                to[i] = pack_half(e0, e1);
                                if (kFine) rest[i] = left_of(to[i], e0, e1);
                            }
                        };
                        fence_loaded(x);
                        tmem_ld_32(col_s + 32, y);
                        weights(x, p, p_rest);
                        fence_loaded(y);
                        weights(y, r, r_rest);
                        float sum[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float2 h = each_of(s2[k]);
                            sum[k] = h.x + h.y;
                        }
                        const float total = (sum[0] + sum[1]) + (sum[2] + sum[3]);
                        fits = __all_sync(0xffffffffu, total <= kHalfMost && vmost <= cref && (have || !live));
                        if (fits) {
                            tmem_st_16(col_s, p);
                            tmem_st_16(col_s + 16, r);
                            if (kFine) {
                                tmem_st_16(col_s + 32, p_rest);
                                tmem_st_16(col_s + 48, r_rest);
                            }
                            // the group's weight out of its sum again
                            if (even) {
                                l = fmaf(total, exp2_fast(-lw[0]), l);
                            } else {
#pragma unroll
                                for (int k = 0; k < 4; ++k) l = fmaf(sum[k], exp2_fast(-lw[k]), l);
                            }
                        }
                    }
                    if (__builtin_expect(!fits, 0)) {
                        uint32_t v[64];
                        // c grows to the scales' range: the same in every row
                        float vmost = 0.0f;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float vs = sm.scale[at][k].y;
                            vmost = vs <= 3.402823466e38f ? fmaxf(vmost, vs) : vmost;
                        }
                        if (vmost > cref) {
                            const float to = __int_as_float(min((__float_as_int(vmost) & 0x7f800000) + (1 << 23), 0x7f000000));
                            if (st > 0 && !(ok = rescale(st + 1 == steps, cref / to))) break;
                            cref = to;
                            logc = static_cast<float>((__float_as_int(to) >> 23) - 127);
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            weigh(sm.scale[at][k], whole || (tok0 + 16 * k < sees && ((valid >> k) & 1u)), fk[k], lw[k]);
                        ptx::tmem_ld_32x2(col_s, col_s + 32, *reinterpret_cast<uint32_t(*)[32]>(v),
                                          *reinterpret_cast<uint32_t(*)[32]>(v + 32));
                        if (!whole) {
                            const int left = sees - tok0;
#pragma unroll
                            for (int j = 0; j < 64; ++j) {
                                const int tok = (j & 7) * 8 + (j >> 3);
                                const bool seen = tok < left && ((valid >> (tok >> 4)) & 1u);
                                v[j] = seen ? v[j] : 0xff800000u;
                            }
                        }
                        float top = -INFINITY;  // log2 of the largest weight
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            minus[k] = lw[k] - ref;
                            float g = -INFINITY;
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                g = fmaxf(fmaxf(g, __uint_as_float(v[2 * k + 8 * i])), __uint_as_float(v[2 * k + 8 * i + 1]));
                            top = fmaxf(top, fmaf(g, fk[k], minus[k]));
                        }
                        // a weight near the end of fp16's range: the row's reference moves, by a power of two, exact
                        // for what has been summed and rounded (64 weights below the limit fit together)
                        const bool moves = top > (have ? kLogLimit : -INFINITY);
                        if (__any_sync(0xffffffffu, moves)) {
                            float keep = 1.0f;
                            if (moves) {
                                const float to = ref + (ceilf(top) - kLogStart);
                                keep = have ? exp2_fast(ref - to) : 0.0f;
                                ref = to;
                                l *= keep;
                                have = true;
                            }
                            if (st > 0 && !(ok = rescale(st + 1 == steps, keep))) break;
#pragma unroll
                            for (int k = 0; k < 4; ++k) minus[k] = lw[k] - ref;
                        }
                        float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            uint32_t p[16], rest[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                const int j = 32 * c + 2 * i, k = i & 3;
                                const float e0 = exp2_fast(fmaf(__uint_as_float(v[j]), fk[k], minus[k]));
                                const float e1 = exp2_fast(fmaf(__uint_as_float(v[j + 1]), fk[k], minus[k]));
                                sum[k] += e0 + e1;
                                p[i] = pack_half(e0, e1);
                                if (kFine) rest[i] = left_of(p[i], e0, e1);
                            }
                            tmem_st_16(col_s + 16 * c, p);
                            if (kFine) tmem_st_16(col_s + 32 + 16 * c, rest);
                        }
#pragma unroll
                        for (int k = 0; k < 4; ++k) l = fmaf(sum[k], exp2_fast(-lw[k]), l);
                    }
                }
                ptx::tmem_wait_st();
                ptx::tc_fence_before();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(smem_u32(&sm.p_full[s][b]));
                ++count;
            }
            if (!ok) break;
            // the odd tiles' sums go to the even ones', through columns of stream 1's scores: its next ones wait
            const bool join = !two && tiles > 1;
            float next_factor = 0.0f;
            if (more && !(join && s == 1)) next_factor = convert();
            if (steps > 0) {
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(smem_u32(&sm.o_full[s]), o_phase, err));
                o_phase ^= 1;
                if (steps > 1) {
                    ok = ok && __all_sync(0xffffffffu, ptx::mbar_wait(smem_u32(&sm.o_most[s]), most_phase, err));
                    most_phase ^= 1;
                }
                if (!ok) break;
                ptx::tc_fence_after();
            }
            // ---- the segment's end
            if (tiles > 0) {
                const bool begins = w.t0 == 0, ends = w.t1 == w.x.tiles, cut = !(begins && ends);
                const bool nan = *reinterpret_cast<volatile int*>(&sm.nan_seen) != 0;
                if (l == 0.0f) ref = kNothing;
                if (s == 1 && !two) {
                    if (join) {
                        // stream 0's warp of the same rows reads this stream's O, and beside it, in the columns of
                        // scores that are no longer needed, its maximum, sum and scale
                        uint32_t x[16] = {__float_as_uint(ref), __float_as_uint(l), __float_as_uint(cref * 0.0078125f), nan_scale};
                        tmem_st_16(tmem + lanes + kColS + 128, x);
                        ptx::tmem_wait_st();
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(smem_u32(&sm.merge_full));
                        ok = __all_sync(0xffffffffu, ptx::mbar_wait(smem_u32(&sm.merge_empty), merge_phase, err));
                        merge_phase ^= 1;
                        if (!ok) break;
                        ptx::tc_fence_after();
                    }
                } else {
                    float f0 = cref * 0.0078125f, f1 = 0.0f, m = ref;  // 2^-7 c
                    const int slot = 2 * blockIdx.x + (begins ? 1 : 0);
                    float* const piece = pieces + static_cast<int64_t>(slot) * piece_rows * (DP + 4);
                    const int64_t t = w.x.r.row0 + i;
                    if (join) {
                        ok = __all_sync(0xffffffffu, ptx::mbar_wait(smem_u32(&sm.merge_full), merge_phase, err));
                        merge_phase ^= 1;
                        if (!ok) break;
                        ptx::tc_fence_after();
                        uint32_t x[16];
                        ptx::tmem_ld_16(tmem + lanes + kColS + 128, x);
                        const float m1 = __uint_as_float(x[0]), l1 = __uint_as_float(x[1]);
                        m = fmaxf(ref, m1);
                        const float k0 = exp2_fast(ref - m), k1 = exp2_fast(m1 - m);
                        // a side without weights has no part; NaN sums stay
                        f0 = l == 0.0f ? 0.0f : f0 * k0;
                        f1 = l1 == 0.0f ? 0.0f : __uint_as_float(x[2]) * k1;
                        nan_scale = nan_scale || x[3];
                        l = (l == 0.0f ? 0.0f : l * k0) + (l1 == 0.0f ? 0.0f : l1 * k1);
                    }
                    const float g = cut ? 1.0f : (l == 0.0f ? 0.0f : 1.0f / l);
                    if (__all_sync(0xffffffffu, !live || (l != 0.0f && !nan_scale)) && !nan) {
                        // nothing special in any row (what runs once an item costs its instructions' fetch: few of them)
                        const float g0 = f0 * g, g1 = f1 * g;
#pragma unroll 1
                        for (int c = 0; c < DP / 16; ++c) {
                            uint32_t v[16], y[16];
                            float f[16];
                            if (join) {
                                ptx::tmem_ld_16x2(col_o + 16 * c, col_o + 128 + 16 * c, v, y);
#pragma unroll
                                for (int j = 0; j < 16; ++j) f[j] = fmaf(__uint_as_float(y[j]), g1, __uint_as_float(v[j]) * g0);
                            } else {
                                ptx::tmem_ld_16(col_o + 16 * c, v);
#pragma unroll
                                for (int j = 0; j < 16; ++j) f[j] = __uint_as_float(v[j]) * g0;
                            }
                            if (live && cut) {
                                float4* const to = reinterpret_cast<float4*>(piece) + 4 * c * piece_rows + in_item;
#pragma unroll
                                for (int j = 0; j < 4; ++j) to[j * piece_rows] = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
                            } else if (live && 16 * c < a.dim) {
                                store(a.out, t * a.out_token_stride + h * a.out_head_stride + 16 * c, f, bf16, out_wide);
                            }
                        }
                    } else
#pragma unroll 1
                    for (int c = 0; c < DP / 16; ++c) {
                        uint32_t v[16], y[16];
                        if (join) ptx::tmem_ld_16x2(col_o + 16 * c, col_o + 128 + 16 * c, v, y);
                        else ptx::tmem_ld_16(col_o + 16 * c, v);
                        const int d = 16 * c;
                        float f[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            float o = f0 == 0.0f ? 0.0f : __uint_as_float(v[j]) * f0;
                            if (join && f1 != 0.0f) o = fmaf(__uint_as_float(y[j]), f1, o);
                            f[j] = nan_scale ? __int_as_float(0x7fffffff) : o * g;
                        }
                        if (nan && live && d < a.dim) {
                            // NaN codes that were set apart: those of tokens that this row sees
                            uint32_t hit = 0;
                            for (int pos = max(all_see, w.t0 * kTok); pos < min(min(sees, w.x.r.length), w.t1 * kTok); ++pos) {
                                const int pg = a.table[w.x.b * a.stride + (pos >> a.page_shift)];
                                if (pg < 0 || pg >= a.pages) continue;
                                const uint4 x = *reinterpret_cast<const uint4*>(
                                    a.v_cache + (((static_cast<int64_t>(pg) * a.heads + w.x.head) << a.page_shift) +
                                                 (pos & (page_size - 1))) * a.dim + d);
                                const uint32_t e[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                                for (int k = 0; k < 4; ++k) {
                                    const uint32_t is = __vcmpeq4(e[k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                                    hit |= ((is & 1u) | ((is >> 7) & 2u) | ((is >> 14) & 4u) | ((is >> 21) & 8u)) << (4 * k);
                                }
                            }
#pragma unroll
                            for (int j = 0; j < 16; ++j)
                                if ((hit >> j) & 1u) f[j] = __int_as_float(0x7fffffff);
                        }
                        if (live && cut) {
                            float4* const to = reinterpret_cast<float4*>(piece) + 4 * c * piece_rows + in_item;
#pragma unroll
                            for (int j = 0; j < 4; ++j) to[j * piece_rows] = make_float4(f[4 * j], f[4 * j + 1], f[4 * j + 2], f[4 * j + 3]);
                        } else if (live && d < a.dim) {
                            store(a.out, t * a.out_token_stride + h * a.out_head_stride + d, f, bf16, out_wide);
                        }
                    }
                    if (join) {
                        ptx::tc_fence_before();
                        __syncwarp();
                        if (lane == 0) ptx::mbar_arrive(smem_u32(&sm.merge_empty));
                    }
                    if (live && cut) {
                        float* const sums = piece + static_cast<int64_t>(piece_rows) * DP + 2 * in_item;
                        sums[0] = m;
                        sums[1] = l;
                    } else if (live && a.lse) {
                        a.lse[t * a.q_heads + h] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
                    }
                    if (cut && row == 0 && s == 0)
                        infos[slot] = PieceInfo{w.x.b, w.x.head, w.x.item, begins, ends};
                }
                ptx::tc_fence_before();
            }
            n += tiles;
            if (w.last) break;
            if (more && join && s == 1) next_factor = convert();
            factor = next_factor;
            w.next(a, group);
        }
    }

    // Tensor memory is given back once every warp has done with it.
    ptx::tc_fence_before();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(smem_u32(&sm.exit_bar));
    if (warp == kMma) {
        __syncwarp();
        ptx::mbar_wait(smem_u32(&sm.exit_bar), 0, err);
        ptx::tc_fence_after();
        ptx::tmem_dealloc(tmem, 512);
    }
}

// One block for each block of the first launch: if it left the first piece of
// an item that goes on, all of the item's pieces are joined here, in order.
template <int DP>
__global__ void __launch_bounds__(256) attention_wide_join(const AttentionArgs a, int blocks, const PieceInfo* infos,
                                                           const float* pieces, int piece_rows, int out_wide) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const PieceInfo info = infos[2 * blockIdx.x + 1];
    if (info.request < 0 || info.ends) return;
    const int group = a.q_heads / a.heads;
    Item x;
    x.r = request_of(a, info.request);
    x.item = info.item;
    shape(x, group);
    int last = blockIdx.x + 1;
    while (last < blocks - 1 && !infos[2 * last].ends) ++last;
    const int64_t size = static_cast<int64_t>(piece_rows) * (DP + 4), ml_at = static_cast<int64_t>(piece_rows) * DP;
    for (int k = blockIdx.y * 256 + threadIdx.x; k < x.rows * (a.dim / 16); k += gridDim.y * 256) {
        const int d = k / x.rows * 16, row = k - d / 16 * x.rows;  // neighbouring threads: neighbouring rows
        auto piece = [&](int c) { return pieces + (c == static_cast<int>(blockIdx.x) ? 2 * c + 1 : 2 * c) * size; };
        auto holds = [&](int c) { return c == static_cast<int>(blockIdx.x) || infos[2 * c].request >= 0; };
        float m = -INFINITY;
        for (int c = blockIdx.x; c <= last; ++c)
            if (holds(c)) m = fmaxf(m, piece(c)[ml_at + 2 * row]);
        const float base = m == -INFINITY ? 0.0f : m;
        float l = 0.0f, f[16] = {};
        for (int c = blockIdx.x; c <= last; ++c) {
            if (!holds(c)) continue;
            const float* const p = piece(c);
            const float lc = p[ml_at + 2 * row + 1];
            if (lc == 0.0f) continue;
            const float g = exp2_fast(p[ml_at + 2 * row] - base);
            l = fmaf(lc, g, l);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float4 u = reinterpret_cast<const float4*>(p)[(d / 4 + j) * piece_rows + row];
                f[4 * j] = fmaf(u.x, g, f[4 * j]);
                f[4 * j + 1] = fmaf(u.y, g, f[4 * j + 1]);
                f[4 * j + 2] = fmaf(u.z, g, f[4 * j + 2]);
                f[4 * j + 3] = fmaf(u.w, g, f[4 * j + 3]);
            }
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
        for (int j = 0; j < 16; ++j) f[j] *= inv;
        const int rr = info.item * kItemRows + row;
        const int64_t t = x.r.row0 + rr / group;
        const int h = info.head * group + rr % group;
        store(a.out, t * a.out_token_stride + h * a.out_head_stride + d, f, a.dtype == kBF16, out_wide);
        if (d == 0 && a.lse) a.lse[t * a.q_heads + h] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
    }
}

// The bytes that every row begins at a multiple of: 32, 16, or 2 for anything else.
int wide_rows(const void* p, int64_t token, int64_t head) {
    const uintptr_t all = reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(token * 2) | static_cast<uintptr_t>(head * 2);
    return all % 32 == 0 ? 32 : all % 16 == 0 ? 16 : 2;
}

size_t round16(size_t n) { return (n + 15) & ~static_cast<size_t>(15); }

int piece_rows_of(int64_t rows, int64_t group) {
    return static_cast<int>(rows * group < kItemRows ? (rows * group + 3) & ~int64_t(3) : kItemRows);
}

template <int DP, bool kFine>
cudaError_t launch(const AttentionArgs& a, cudaStream_t stream) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const int blocks = device_info(dev).sm_count;
    Maps maps;
    const uint32_t page = 1u << a.page_shift;
    const uint64_t dims[3] = {static_cast<uint64_t>(a.dim), static_cast<uint64_t>(a.heads) * page,
                              static_cast<uint64_t>(a.pages > 0 ? a.pages : 1)};
    const uint64_t strides[2] = {static_cast<uint64_t>(a.dim), static_cast<uint64_t>(a.heads) * page * a.dim};
    const uint32_t box[3] = {DP, page < 64 ? page : 64, 1};
    // a cache without pages: nothing is loaded, but a map needs an address
    const void* const k = a.pages > 0 ? a.k_cache : a.workspace;
    const void* const v = a.pages > 0 ? a.v_cache : a.workspace;
    if (!encode_tmap_bytes(&maps.k, k, dims, strides, box) || !encode_tmap_bytes(&maps.v, v, dims, strides, box))
        return cudaErrorInvalidValue;
    uint8_t* const w = static_cast<uint8_t*>(a.workspace);
    PieceInfo* const infos = reinterpret_cast<PieceInfo*>(w);
    float* const pieces = reinterpret_cast<float*>(w + round16(sizeof(PieceInfo) * 2 * blocks));
    const int piece_rows = piece_rows_of(a.rows, a.q_heads / a.heads);
    const size_t smem = sizeof(Smem<DP>) + 1024;
    static std::atomic<uint64_t> allowed{0};
    e = allow_shared(attention_wide_kernel<DP, kFine>, smem, dev, allowed);
    if (e != cudaSuccess) return e;
    const bool q_wide = wide_rows(a.q, a.q_token_stride, a.q_head_stride) >= 16;
    const int out_wide = wide_rows(a.out, a.out_token_stride, a.out_head_stride);
    attention_wide_kernel<DP, kFine><<<blocks, kThreads, smem, stream>>>(a, maps, device_error_word(), infos, pieces,
                                                                  piece_rows, q_wide, out_wide);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks, 4);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attention_wide_join<DP>, a, blocks, static_cast<const PieceInfo*>(infos),
                              static_cast<const float*>(pieces), piece_rows, out_wide);
}

}  // namespace

size_t attention_wide_workspace(int64_t rows, int64_t group, int64_t dim, int sms) {
    return round16(sizeof(PieceInfo) * 2 * sms) +
           sizeof(float) * 2 * sms * static_cast<size_t>(piece_rows_of(rows, group)) * ((dim <= 64 ? 64 : 128) + 4);
}

cudaError_t launch_attention_wide(const AttentionArgs& a, cudaStream_t stream) {
    if (a.dtype == kBF16) return a.dim <= 64 ? launch<64, false>(a, stream) : launch<128, false>(a, stream);
    return a.dim <= 64 ? launch<64, true>(a, stream) : launch<128, true>(a, stream);
}

}  // namespace lik
