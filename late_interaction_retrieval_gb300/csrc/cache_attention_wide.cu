// cache_attention_wide.cu -- attention over the 8-bit cache for many rows a
// key head (drafts of grouped heads, prompts): the products on tcgen05.
//
// A tile is 128 tokens against 128 rows: S = Q K^T in tensor memory, its
// softmax weights back into tensor memory as fp16, O += P V.  Two tiles are in
// work at a time, in two streams with a softmax warpgroup, an S/P and an O
// accumulator each, so that the tensor cores work on one while the other's
// exponentials are taken.  Where an item has more than 128 rows the streams
// are its two halves, on the same tokens (the codes are widened once for
// both); else they are the even and the odd tiles of the same rows, joined at
// the item's end.
//
// The codes become fp16 (exactly) on their way from the TMA ring to the MMA's
// operand tiles.  K stays token by token.  V is transposed, so that both
// operands are K-major: a thread takes 8 tokens of 8 dimensions, byte
// permutes pair the tokens, and every store is 16 bytes.  Those 8 tokens lie
// 8 apart in a block of 64 (which keeps the loads free of bank conflicts), so
// the tokens of S's columns are ordered that way: column j of a block holds
// token (j mod 8) * 8 + j / 8.
//
// The weights are 2^7 exp2(z - m) (the page's scale / c), with a maximum m
// that is only moved when it is exceeded by 2^8 and a scale c that is moved to
// twice the largest; both moves rescale O, and are rare.  Work is spread as
// in the kernel for few rows: the batch's tiles end to end, one equal range a
// block, pieces of cut items joined by a second launch.
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
    uint64_t o_step[2], o_full[2];  // a step is in O; an item's last one is
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
    const int sees = x.r.length - x.r.n + (first + x.rows - 1) / group + 1;
    x.tiles = max(1, (sees + kTok - 1) / kTok);
}

__device__ __forceinline__ long long steps_of(const Request& r, int group, int i) {
    Item x;
    x.r = r;
    x.item = i;
    shape(x, group);
    return static_cast<long long>(x.tiles) * (x.two ? 2 : 1);
}

__device__ long long steps_of_head(const Request& r, int group) {
    long long s = 0;
    for (int i = 0; i < items_of(r, group); ++i) s += steps_of(r, group, i);
    return s;
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

// 64 columns of this thread's lane, and their maximum, which the loads take
// (loads and wait in one statement, so that no use comes before the wait).
__device__ __forceinline__ void tmem_ldmax_64(uint32_t taddr, uint32_t (&v)[64], float& mx) {
    float a, b, c, d;
    asm volatile(
        "tcgen05.ld.red.sync.aligned.32x32b.x16.max.f32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, %64, [%68];\n\t"
        "tcgen05.ld.red.sync.aligned.32x32b.x16.max.f32 {%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, %65, [%69];\n\t"
        "tcgen05.ld.red.sync.aligned.32x32b.x16.max.f32 {%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47}, %66, [%70];\n\t"
        "tcgen05.ld.red.sync.aligned.32x32b.x16.max.f32 {%48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, %67, [%71];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
          "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
          "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
          "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31]),
          "=r"(v[32]), "=r"(v[33]), "=r"(v[34]), "=r"(v[35]), "=r"(v[36]), "=r"(v[37]), "=r"(v[38]), "=r"(v[39]),
          "=r"(v[40]), "=r"(v[41]), "=r"(v[42]), "=r"(v[43]), "=r"(v[44]), "=r"(v[45]), "=r"(v[46]), "=r"(v[47]),
          "=r"(v[48]), "=r"(v[49]), "=r"(v[50]), "=r"(v[51]), "=r"(v[52]), "=r"(v[53]), "=r"(v[54]), "=r"(v[55]),
          "=r"(v[56]), "=r"(v[57]), "=r"(v[58]), "=r"(v[59]), "=r"(v[60]), "=r"(v[61]), "=r"(v[62]), "=r"(v[63]),
          "=f"(a), "=f"(b), "=f"(c), "=f"(d)
        : "r"(taddr), "r"(taddr + 16), "r"(taddr + 32), "r"(taddr + 48)
        : "memory");
    mx = fmaxf(fmaxf(a, b), fmaxf(c, d));
}

// Registers of a warpgroup's threads: 256 threads of 144 and 384 of 64 are the
// 640 of 96 that the block is launched with.
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 144;"); }
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 64;"); }

// 8 neighbouring dimensions of one row to the output.
__device__ __forceinline__ void store8(void* out, int64_t at, const float (&f)[8], bool bf16, bool wide) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (bf16) {
            const __nv_bfloat162 x = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&x);
        } else {
            w[i] = pack_half(f[2 * i], f[2 * i + 1]);
        }
    }
    uint16_t* const p = static_cast<uint16_t*>(out) + at;
    if (wide) {
        *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            p[2 * i] = static_cast<uint16_t>(w[i]);
            p[2 * i + 1] = static_cast<uint16_t>(w[i] >> 16);
        }
    }
}

template <int DP>
__global__ void __launch_bounds__(kThreads, 1)
    attention_wide_kernel(const AttentionArgs a, const __grid_constant__ Maps maps, unsigned int* err,
                          PieceInfo* infos, float* pieces, int piece_rows, bool q_wide, bool out_wide) {
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
            ptx::mbar_init(smem_u32(&sm.o_step[i]), 1);
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
    // ---- the block's range of steps (a tile of one stream), from every request's
    const int B = a.requests, each = (B + kThreads - 1) / kThreads;
    long long mine = 0;
    for (int b = min(tid * each, B); b < min(tid * each + each, B); ++b)
        mine += steps_of_head(request_of(a, b), group) * a.heads;
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) sm.warp_sum[warp] = incl;
    __syncthreads();
    long long all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) incl += sm.warp_sum[w];
        all += sm.warp_sum[w];
    }
    const long long excl = incl - mine;
    // a block has two steps at least
    const long long active = max(1ll, min(static_cast<long long>(gridDim.x), all / 2));
    const long long u0 = blockIdx.x < active ? all * blockIdx.x / active : all;
    const long long u1 = blockIdx.x < active ? all * (blockIdx.x + 1) / active : all;
    if (tid < 2) infos[2 * blockIdx.x + tid] = PieceInfo{-1, 0, 0, 0, 0};
    if (u0 >= u1) return;
    // the tile that holds step u, by the thread whose requests do; a range ends
    // before the tile of its last bound, or behind the batch's last
    auto locate = [&](long long u, int* to, int more) {
        if (u < excl || u >= incl) return;
        long long rest = u - excl;
        int b = tid * each;
        Request r = request_of(a, b);
        long long per = steps_of_head(r, group);
        while (rest >= per * a.heads) {
            rest -= per * a.heads;
            r = request_of(a, ++b);
            per = steps_of_head(r, group);
        }
        to[0] = b;
        to[1] = static_cast<int>(rest / per);
        rest %= per;
        int i = 0;
        while (rest >= steps_of(r, group, i)) rest -= steps_of(r, group, i++);
        Item x;
        x.r = r;
        x.item = i;
        shape(x, group);
        to[2] = i;
        to[3] = static_cast<int>(x.two ? rest / 2 : rest) + more;
    };
    locate(u0, sm.start, 0);
    if (u1 < all) locate(u1, sm.end, 0);
    else locate(all - 1, sm.end, 1);
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
            const int all_see = w.x.r.length - w.x.r.n + (w.x.item * kItemRows) / group + 1;
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
#pragma unroll 2
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
        if (lane == 0) {
            constexpr uint32_t kIdS = ptx::f16_idesc(kM, kTok, false), kIdO = ptx::f16_idesc(kM, DP, false);
            const int s = warp - kMma;
            const uint32_t col_s = tmem + kColS + 128 * s, col_o = tmem + kColO + 128 * s;
            int n = 0;                    // tiles before this segment
            int scored = 0, summed = 0;   // steps of this stream so far
            uint32_t q_phase = 0;
            while (ok) {
                const bool two = w.x.two;
                const int tiles = w.t1 - w.t0, steps = two ? tiles : (tiles + 1 - s) / 2;
                // A buffer is empty again when both streams have done with it; a tile of one stream counts twice.
                auto done = [&](uint64_t* bar) {
                    ptx::mma_commit(smem_u32(bar));
                    if (!two) ptx::mma_commit(smem_u32(bar));
                };
                // Step i's tile.  Tiles are filled in order, so the other stream's phase between two of this
                // stream's in one buffer has been completed when this one asks for the second.
                auto tile_of = [&](int i) { return n + (two ? i : 2 * i + s); };
                auto score = [&](int i) {
                    const int t = tile_of(i), kb = t % kKeys, b = scored & 1;
                    ok = ok && ptx::mbar_wait(smem_u32(&sm.k_full[kb]), (t / kKeys) & 1, err);
                    if (!ok) return;
                    ptx::tc_fence_after();
                    // the buffer's weights of two steps ago were multiplied by an instruction before this one
                    uint64_t qd = ptx::sw128_kmajor_desc(smem_u32(sm.q[s][0]));
                    uint64_t kd = ptx::sw128_kmajor_desc(smem_u32(sm.k[kb][0]));
#pragma unroll 1
                    for (int atom = 0; atom < DP / 64; ++atom) {  // 64 dimensions: 4 steps of 32 bytes
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            ptx::mma_f16(col_s + 64 * b, qd + 2 * k, kd + 2 * k, kIdS, atom > 0 || k != 0);
                        qd += kM * 128 / 16;
                        kd += kTok * 128 / 16;
                    }
                    ptx::mma_commit(smem_u32(&sm.s_full[s][b]));
                    done(&sm.k_empty[kb]);
                    ++scored;
                };
                if (steps > 0) {
                    ok = ptx::mbar_wait(smem_u32(&sm.q_full[s]), q_phase, err);
                    q_phase ^= 1;
                }
                for (int i = 0; ok && i < min(kAhead, steps); ++i) score(i);
                for (int i = 0; ok && i < steps; ++i) {
                    const int t = tile_of(i), vb = t & (kValues - 1), b = summed & 1;
                    ok = ptx::mbar_wait(smem_u32(&sm.v_full[vb]), (t / kValues) & 1, err) &&
                         ptx::mbar_wait(smem_u32(&sm.p_full[s][b]), (summed >> 1) & 1, err);
                    if (!ok) break;
                    ++summed;
                    ptx::tc_fence_after();
                    const uint64_t vd = ptx::sw128_kmajor_desc(smem_u32(sm.v[vb]));
#pragma unroll
                    for (int k = 0; k < kTok / 16; ++k)
                        mma_f16_ts(col_o, col_s + 64 * b + 8 * k, vd + 2 * k, kIdO, i > 0 || k != 0);
                    ptx::mma_commit(smem_u32(&sm.o_step[s]));
                    if (i + 1 == steps) ptx::mma_commit(smem_u32(&sm.o_full[s]));
                    done(&sm.v_empty[vb]);
                    if (i + kAhead < steps) score(i + kAhead);
                }
                n += tiles;
                if (!ok || w.last) break;
                w.next(a, group);
            }
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
        int n = 0, count = 0;  // tiles, and steps of this stream, before
        uint32_t o_phase = 0, merge_phase = 0;
        while (ok) {
            const bool two = w.x.two;
            const int tiles = w.t1 - w.t0, steps = two ? tiles : (tiles + 1 - s) / 2;
            const int in_item = (two ? s * kM : 0) + row;
            const bool live = in_item < w.x.rows;
            const int rr = w.x.item * kItemRows + in_item;  // of the request's rows
            const int i = live ? rr / group : 0;
            const int h = w.x.head * group + (live ? rr % group : 0);
            const int sees = live ? w.x.r.length - w.x.r.n + i + 1 : 0;
            const int all_see = w.x.r.length - w.x.r.n + (w.x.item * kItemRows) / group + 1;
            const bool idle = __ballot_sync(0xffffffffu, live) == 0;  // no row of this warp's: its weights do not matter
            float factor = 0.0f, ref = kNothing, l = 0.0f, cref = 0.0f, logc = -127.0f;  // logc: log2 of cref
            bool nan_scale = false;  // the row sees a page whose values' scale is not finite
            if (steps > 0) {
                // the row of q, scaled to fp16's range
                const uint16_t* const src = static_cast<const uint16_t*>(a.q) + (w.x.r.row0 + i) * a.q_token_stride +
                                            h * a.q_head_stride;
                auto load = [&](int c) {  // 8 dimensions
                    if (!live || c * 8 >= a.dim) return make_uint4(0, 0, 0, 0);
                    if (q_wide) return __ldg(reinterpret_cast<const uint4*>(src) + c);
                    uint32_t e[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        e[k] = src[8 * c + 2 * k] | (static_cast<uint32_t>(src[8 * c + 2 * k + 1]) << 16);
                    return make_uint4(e[0], e[1], e[2], e[3]);
                };
                // two passes of little code (what runs once an item is fetched each time), the second from L1
                float most = 0.0f;
#pragma unroll 1
                for (int c = 0; c < DP / 8; c += 8) {
                    uint4 x[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[k] = load(c + k);
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        const float2 f = widen_q(reinterpret_cast<const uint32_t*>(x)[k], bf16);
                        most = fmaxf(most, fmaxf(fabsf(f.x), fabsf(f.y)));
                    }
                }
                const int shift = row_shift(most);
                const float2 up = power_of_two(shift), down = power_of_two(-shift);
#pragma unroll 1
                for (int c = 0; c < DP / 8; c += 4) {
                    uint4 x[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) x[k] = load(c + k);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t* const e = reinterpret_cast<const uint32_t*>(&x[k]);
                        uint32_t o[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const float2 f = widen_q(e[j], bf16);
                            o[j] = pack_half(f.x * up.x * up.y, f.y * up.x * up.y);
                        }
                        sts16(smem_u32(sm.q[s][(c + k) >> 3]) + tile_at(row, (c + k) & 7), o[0], o[1], o[2], o[3]);
                    }
                }
                factor = a.scale * 1.44269504088896341f * down.x * down.y;
                fence_operands();
                __syncwarp();
                if (lane == 0) ptx::mbar_arrive(smem_u32(&sm.q_full[s]));
            }
            // O times `keep` (1 in rows that need none).  It is at rest once the step before is in it: this step's
            // product waits for its weights.  (The step before that is: this step's scores came after it.  So the
            // phase is not taken for one of two steps ago.)
            auto rescale = [&](float keep) {
                if (!__all_sync(0xffffffffu, ptx::mbar_wait(smem_u32(&sm.o_step[s]), (count - 1) & 1, err))) return false;
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
                if (!idle) {
                    const uint32_t valid = sm.valid[at];
                    const bool whole = tok0 + kTok <= all_see && valid == 15u;
                    const bool even = whole && page_size >= 64;  // one page, no token hidden
                    // 16 tokens that share their scales: the columns with (j mod 8) / 2 alike
                    uint32_t v[64];
                    float fk[4], lw[4], mx = 0.0f;
                    // c grows to the scales' range: the same in every row
                    auto grow = [&](float vmost) {
                        const float to = __int_as_float(min((__float_as_int(vmost) & 0x7f800000) + (1 << 23), 0x7f000000));
                        if (st > 0) ok = rescale(cref / to);
                        cref = to;
                        logc = static_cast<float>((__float_as_int(to) >> 23) - 127);
                    };
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
                    if (even) {
                        const float4 x = sm.scale[at][0];
                        tmem_ldmax_64(col_s, v, mx);
                        if (x.y > cref && x.y <= 3.402823466e38f) grow(x.y);
                        weigh(x, true, fk[0], lw[0]);
#pragma unroll
                        for (int k = 1; k < 4; ++k) {
                            fk[k] = fk[0];
                            lw[k] = lw[0];
                        }
                    } else {
                        float vmost = 0.0f;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float vs = sm.scale[at][k].y;
                            vmost = vs <= 3.402823466e38f ? fmaxf(vmost, vs) : vmost;
                        }
                        if (vmost > cref) grow(vmost);
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
                    }
                    if (!ok) break;
                    float minus[4];
                    auto limit = [&]() {  // log2 of the largest weight; the groups' terms under the reference
#pragma unroll
                        for (int k = 0; k < 4; ++k) minus[k] = lw[k] - ref;
                        if (even) return fmaf(mx, fk[0], minus[0]);
                        float top = -INFINITY;
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            float g = -INFINITY;
#pragma unroll
                            for (int i = 0; i < 8; ++i)
                                g = fmaxf(fmaxf(g, __uint_as_float(v[2 * k + 8 * i])), __uint_as_float(v[2 * k + 8 * i + 1]));
                            top = fmaxf(top, fmaf(g, fk[k], minus[k]));
                        }
                        return top;
                    };
                    const float top = limit();
                    // a weight beyond fp16's range: the row's reference moves, by a power of two, exact for what has
                    // been summed and rounded
                    if (__any_sync(0xffffffffu, top > kLogTop)) {
                        float keep = 1.0f;
                        if (top > kLogTop) {
                            const float by = ceilf(top) - kLogStart;
                            keep = exp2_fast(-by);  // 0 for the first tokens that a row sees
                            ref += by;
                            l *= keep;
                        }
                        if (st > 0 && !(ok = rescale(keep))) break;
#pragma unroll
                        for (int k = 0; k < 4; ++k) minus[k] = lw[k] - ref;
                    }
                    // the weights take the place of the scores
                    float sum[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t p[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const int j = 32 * c + 2 * i, k = i & 3;
                            const float e0 = exp2_fast(fmaf(__uint_as_float(v[j]), fk[k], minus[k]));
                            const float e1 = exp2_fast(fmaf(__uint_as_float(v[j + 1]), fk[k], minus[k]));
                            sum[k] += e0 + e1;
                            p[i] = pack_half(e0, e1);
                        }
                        tmem_st_16(col_s + 16 * c, p);
                    }
                    // the group's weight out of its sum again
                    if (even) {
                        l = fmaf((sum[0] + sum[1]) + (sum[2] + sum[3]), exp2_fast(-lw[0]), l);
                    } else {
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
            if (steps > 0) {
                ok = __all_sync(0xffffffffu, ptx::mbar_wait(smem_u32(&sm.o_full[s]), o_phase, err));
                o_phase ^= 1;
                if (!ok) break;
                ptx::tc_fence_after();
            }
            // ---- the segment's end
            if (tiles > 0) {
                const bool begins = w.t0 == 0, ends = w.t1 == w.x.tiles, cut = !(begins && ends);
                const bool join = !two && tiles > 1;  // the odd tiles' sums go to the even ones'
                const bool nan = *reinterpret_cast<volatile int*>(&sm.nan_seen) != 0;
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
#pragma unroll 1
                    for (int c = 0; c < DP / 16; ++c) {
                        uint32_t v[16], y[16];
                        if (join) ptx::tmem_ld_16x2(col_o + 16 * c, col_o + 128 + 16 * c, v, y);
                        else ptx::tmem_ld_16(col_o + 16 * c, v);
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int d = 16 * c + 8 * e;
                            float f[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                float o = f0 == 0.0f ? 0.0f : __uint_as_float(v[8 * e + j]) * f0;
                                if (join && f1 != 0.0f) o = fmaf(__uint_as_float(y[8 * e + j]), f1, o);
                                f[j] = nan_scale ? __int_as_float(0x7fffffff) : o * g;
                            }
                            if (nan && live && d < a.dim) {
                                // NaN codes that were set apart: those of tokens that this row sees
                                uint32_t hit = 0;
                                for (int pos = max(all_see, w.t0 * kTok); pos < min(sees, w.t1 * kTok); ++pos) {
                                    const int pg = a.table[w.x.b * a.stride + (pos >> a.page_shift)];
                                    if (pg < 0 || pg >= a.pages) continue;
                                    const uint2 x = *reinterpret_cast<const uint2*>(
                                        a.v_cache + (((static_cast<int64_t>(pg) * a.heads + w.x.head) << a.page_shift) +
                                                     (pos & (page_size - 1))) * a.dim + d);
                                    const uint32_t lo = __vcmpeq4(x.x & 0x7f7f7f7fu, 0x7f7f7f7fu);
                                    const uint32_t hi = __vcmpeq4(x.y & 0x7f7f7f7fu, 0x7f7f7f7fu);
                                    hit |= (lo & 0x01020408u) | (hi & 0x10204080u);
                                }
                                // bytes of lo: bits 3, 10, 17, 24; of hi: 7, 14, 21, 28 (dimension 0 lowest)
#pragma unroll
                                for (int j = 0; j < 8; ++j) {
                                    const int bit = j < 4 ? 3 + 7 * j : 7 + 7 * (j - 4);
                                    if ((hit >> bit) & 1u) f[j] = __int_as_float(0x7fffffff);
                                }
                            }
                            if (live && cut) {
                                float4* const to = reinterpret_cast<float4*>(piece + in_item * DP + d);
                                to[0] = make_float4(f[0], f[1], f[2], f[3]);
                                to[1] = make_float4(f[4], f[5], f[6], f[7]);
                            } else if (live && d < a.dim) {
                                store8(a.out, t * a.out_token_stride + h * a.out_head_stride + d, f, bf16, out_wide);
                            }
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
                                                           const float* pieces, int piece_rows, bool out_wide) {
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
    const int per_row = a.dim / 8;
    for (int k = blockIdx.y * 256 + threadIdx.x; k < x.rows * per_row; k += gridDim.y * 256) {
        const int row = k / per_row, d = (k - row * per_row) * 8;
        auto piece = [&](int c) { return pieces + (c == static_cast<int>(blockIdx.x) ? 2 * c + 1 : 2 * c) * size; };
        float m = -INFINITY;
        for (int c = blockIdx.x; c <= last; ++c) m = fmaxf(m, piece(c)[ml_at + 2 * row]);  // a block has a tile at least
        const float base = m == -INFINITY ? 0.0f : m;
        float l = 0.0f, f[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        for (int c = blockIdx.x; c <= last; ++c) {
            const float* const p = piece(c);
            const float lc = p[ml_at + 2 * row + 1];
            if (lc == 0.0f) continue;
            const float g = exp2_fast(p[ml_at + 2 * row] - base);
            l = fmaf(lc, g, l);
            const float4 u = *reinterpret_cast<const float4*>(p + row * DP + d);
            const float4 v = *reinterpret_cast<const float4*>(p + row * DP + d + 4);
            f[0] = fmaf(u.x, g, f[0]);
            f[1] = fmaf(u.y, g, f[1]);
            f[2] = fmaf(u.z, g, f[2]);
            f[3] = fmaf(u.w, g, f[3]);
            f[4] = fmaf(v.x, g, f[4]);
            f[5] = fmaf(v.y, g, f[5]);
            f[6] = fmaf(v.z, g, f[6]);
            f[7] = fmaf(v.w, g, f[7]);
        }
        const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= inv;
        const int rr = info.item * kItemRows + row;
        const int64_t t = x.r.row0 + rr / group;
        const int h = info.head * group + rr % group;
        store8(a.out, t * a.out_token_stride + h * a.out_head_stride + d, f, a.dtype == kBF16, out_wide);
        if (d == 0 && a.lse) a.lse[t * a.q_heads + h] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
    }
}

bool wide_rows(const void* p, int64_t token, int64_t head) {
    return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(token * 2) | static_cast<uintptr_t>(head * 2)) & 15) == 0;
}

size_t round16(size_t n) { return (n + 15) & ~static_cast<size_t>(15); }

int piece_rows_of(int64_t rows, int64_t group) {
    return static_cast<int>(rows * group < kItemRows ? (rows * group + 3) & ~int64_t(3) : kItemRows);
}

template <int DP>
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
    e = allow_shared(attention_wide_kernel<DP>, smem, dev, allowed);
    if (e != cudaSuccess) return e;
    const bool q_wide = wide_rows(a.q, a.q_token_stride, a.q_head_stride);
    const bool out_wide = wide_rows(a.out, a.out_token_stride, a.out_head_stride);
    attention_wide_kernel<DP><<<blocks, kThreads, smem, stream>>>(a, maps, device_error_word(), infos, pieces,
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
    return a.dim <= 64 ? launch<64>(a, stream) : launch<128>(a, stream);
}

}  // namespace lik
