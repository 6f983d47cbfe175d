// cache_attention_split.cu -- attention over the 8-bit cache for few rows a
// key head (single tokens): the cache is read once, at the memory's rate.
//
// A unit is 32 tokens of one (request, key head, 8 or 16 rows).  The units of
// the batch, laid end to end, are cut into one equal range a block, so that
// long and short requests load the chip evenly; a request that is cut leaves
// partial sums, which a second launch joins in the order of the cache.  In a
// block every warp takes every n-th unit, with a ring of its own that TMA
// fills: no warp waits for another until a request's end.
//
// Products are m16n8k16 with the tokens (scores) and the dimensions (output)
// as M and 8 rows as N, so that no product is spent on rows that are not
// there: S^T = K Q^T, O^T = V^T P^T.  The codes of 8 bits become fp16 in
// registers on their way from shared memory to the fragments (exactly, one
// conversion for two codes), and the order of the dimensions and tokens inside
// a fragment is chosen so that every load is 16 bytes wide: a thread's K codes
// are 32 neighbouring dimensions of one token, its V codes 16 neighbouring
// dimensions of 4 tokens, transposed by byte permutes.  The weights go from
// the one product's layout to the other's by an 8x8 transpose in registers.
//
// Rows are scaled to fp16's range by a power of two.  A softmax weight is
// rounded to fp16 as 2^7 exp(z - ref) * (the page's scale / c): ref is a power
// of two near the row's largest weight, and moves only where one passes 2^15;
// c is a power of two not below the scales.  So a unit needs no maximum over
// the warp, and sums are seldom rescaled, exactly.  11 bits are kept over 20
// binades below the largest weight, 2^-31 of it is lost; for fp16 outputs,
// where that would show, what the rounding left is multiplied too (8% more
// time).  Statistics, sums and the join are fp32.
//
// What bounds it: the latency of a warp's chain (620 instructions a unit at 45%
// of the issue slots; 12 warps an SM are all that the registers hold), not the
// memory: 64 requests of 300007 tokens together, 8 key heads of 128, 4 rows:
// 129 us, 4.8 TB/s (61% of the DRAM's cycles); one request of 131071: 56 us.
#include "cache_attention.h"
#include "tmap.h"

namespace lik {
namespace {

using namespace attn;

constexpr int kTok = 32;  // tokens of a unit

// Blocks of 8 rows (NR of them), warps of a block and stages of a warp's ring:
// 16 rows need more registers, so fewer warps with deeper rings.
template <int NR>
struct Shape;
template <>
struct Shape<1> {
    static constexpr int kWarps = 12, kStages = 2;
};
template <>
struct Shape<2> {
    static constexpr int kWarps = 8, kStages = 3;
};

// Where a block's pieces of cut requests lie, and whose they are.
struct PieceInfo {
    int request, unit;  // unit: head * row tiles + row tile; request -1: no piece
    int begins, ends;   // whether it holds the first / the last tokens
};
template <int DP, int NR>
struct Piece {
    float m[8 * NR], l[8 * NR];
    float4 o[8 * NR * DP / 4];
};

template <int DP, int NR>
struct Smem {
    static constexpr int kWarps = Shape<NR>::kWarps, kStages = Shape<NR>::kStages;
    static constexpr int kTile = kTok * DP;  // bytes of one operand's tile
    alignas(1024) uint8_t ring[kWarps][kStages][2][kTile];
    float4 join[kWarps][4][32];  // 4 vectors of every lane's sums at a time
    float m[kWarps][8 * NR], l[kWarps][8 * NR], c[kWarps];
    alignas(16) float scale[kWarps][kStages][4];  // keys' and values' of the first 16 tokens, of the last 16
    uint64_t full[kWarps][kStages];
    int2 page[kWarps][kStages];
    long long warp_sum[kWarps];
};

struct Maps {
    CUtensorMap k, v;
};

// A request's units.
struct Span {
    Request r;
    int tiles, row_tiles;
    __device__ __forceinline__ long long units(int heads) const {
        return static_cast<long long>(tiles) * row_tiles * heads;
    }
};

template <int NR>
__device__ __forceinline__ Span span_of(const AttentionArgs& a, int b, int group) {
    Span s;
    s.r = request_of(a, b);
    s.tiles = s.r.n ? max(1, (s.r.length + kTok - 1) / kTok) : 0;
    s.row_tiles = (s.r.n * group + 8 * NR - 1) / (8 * NR);
    return s;
}

// A place in the order of units: requests, key heads, row tiles, tiles.
struct Cursor {
    int b, head, row_tile, tile;
    Span s;
};

template <int NR>
__device__ __forceinline__ void settle(const AttentionArgs& a, Cursor& c, int group) {
    while (c.tile >= c.s.tiles) {
        c.tile -= c.s.tiles;
        if (++c.row_tile < c.s.row_tiles) continue;
        c.row_tile = 0;
        if (++c.head < a.heads) continue;
        c.head = 0;
        do {
            if (++c.b >= a.requests) {
                c.s.tiles = INT32_MAX;  // behind the last unit
                return;
            }
            c.s = span_of<NR>(a, c.b, group);
        } while (c.s.tiles == 0);
    }
}

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The transpose of an 8x8 matrix of 16-bit elements over the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

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

// Shared memory offset of 16-byte chunk `c` of row `r` in a tile as TMA
// swizzles it: rows of 128 bytes, chunk ^= row mod 8; of 64 bytes, chunk ^=
// (row / 2) mod 4.
template <int DP>
__device__ __forceinline__ uint32_t chunk_at(int r, int c) {
    return DP == 128 ? r * 128 + ((c ^ (r & 7)) << 4) : r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
}

// One row's 4 neighbouring dimensions to the output.
__device__ __forceinline__ void store4(void* out, int64_t at, float4 v, bool bf16, bool wide) {
    uint32_t lo, hi;
    if (bf16) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y), y = __floats2bfloat162_rn(v.z, v.w);
        lo = *reinterpret_cast<const uint32_t*>(&x);
        hi = *reinterpret_cast<const uint32_t*>(&y);
    } else {
        lo = pack_half(v.x, v.y);
        hi = pack_half(v.z, v.w);
    }
    uint16_t* const p = static_cast<uint16_t*>(out) + at;
    if (wide) {
        *reinterpret_cast<uint2*>(p) = make_uint2(lo, hi);
    } else {
        p[0] = static_cast<uint16_t>(lo);
        p[1] = static_cast<uint16_t>(lo >> 16);
        p[2] = static_cast<uint16_t>(hi);
        p[3] = static_cast<uint16_t>(hi >> 16);
    }
}

// Vector k of a lane's sums: 4 of its DP / 8 dimensions of one of its 2 NR rows.
template <int DP>
__device__ __forceinline__ void vector_place(int k, int lane, int& row, int& dim) {
    constexpr int per_row = DP / 32;
    const int e = k / per_row;
    row = (e >> 1) * 8 + (lane & 3) * 2 + (e & 1);
    dim = (lane >> 2) * (DP / 8) + (k % per_row) * 4;
}

template <int DP, int NR>
__device__ __forceinline__ void write_vector(const AttentionArgs& a, const Request& r, int head, int row_tile,
                                             int group, int k, int lane, float4 o, float l, float m, bool wide) {
    int row, dim;
    vector_place<DP>(k, lane, row, dim);
    const int rr = row_tile * 8 * NR + row;
    if (rr >= r.n * group) return;
    const int64_t t = r.row0 + rr / group;
    const int h = head * group + rr % group;
    const float inv = l == 0.0f ? 0.0f : 1.0f / l;
    if (l == 0.0f) o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    o.x *= inv;
    o.y *= inv;
    o.z *= inv;
    o.w *= inv;
    if (dim < a.dim)
        store4(a.out, t * a.out_token_stride + h * a.out_head_stride + dim, o, a.dtype == kBF16, wide);
    if (dim == 0 && a.lse)
        a.lse[t * a.q_heads + h] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.693147180559945309f;
}

template <int DP, int NR, bool kFine>
__global__ void __launch_bounds__(32 * Shape<NR>::kWarps, 1)
    attention_split_kernel(const AttentionArgs a, const __grid_constant__ Maps maps, unsigned int* err,
                           PieceInfo* infos, Piece<DP, NR>* pieces, bool q_wide, bool out_wide) {
    constexpr int kWarps = Shape<NR>::kWarps, kStages = Shape<NR>::kStages, kThreads = 32 * kWarps, kRows = 8 * NR;
    constexpr int KS = DP / 16;    // k-steps of a score, words of K codes a thread and token
    constexpr int MB = DP / 16;    // m-blocks of the output
    constexpr int VW = DP / 32;    // words of V codes a thread and token
    constexpr int VR = DP / 32;    // vectors of a row
    constexpr int kVectors = 2 * NR * VR;
    extern __shared__ uint8_t raw[];
    Smem<DP, NR>& sm = *reinterpret_cast<Smem<DP, NR>*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, q4 = lane & 3;
    const int group = a.q_heads / a.heads;
    const bool bf16 = a.dtype == kBF16;

    if (lane == 0) {
        for (int s = 0; s < kStages; ++s) ptx::mbar_init(ptx::smem_u32(&sm.full[warp][s]), 1);
        ptx::fence_mbar_init();
    }
    // every block sums the requests' units for itself: thread i those of its
    // neighbouring requests
    const int B = a.requests, each = (B + kThreads - 1) / kThreads;
    long long mine = 0;
    for (int b = min(tid * each, B); b < min(tid * each + each, B); ++b) mine += span_of<NR>(a, b, group).units(a.heads);
    long long incl = mine;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, incl, d);
        if (lane >= d) incl += o;
    }
    if (lane == 31) sm.warp_sum[warp] = incl;
    __syncthreads();
    long long units = 0;
    for (int w = 0; w < kWarps; ++w) {
        if (w < warp) incl += sm.warp_sum[w];
        units += sm.warp_sum[w];
    }
    long long* const chunk = reinterpret_cast<long long*>(&sm.join);
    chunk[tid] = incl - mine;
    __syncthreads();

    // A block has a unit at least; blocks without any have no piece.  A block takes its requests one after another, so
    // short ones are spread although most warps then have nothing to do: 24 requests of 515 tokens together take 17 us
    // with a unit a block, 35 with 4, 52 with 8; one of 4000 17, 17, 21 (8 key heads of 128); one of 300, one key head,
    // 15, 15, 13.
    const long long active = max(1ll, min(static_cast<long long>(gridDim.x), units));
    const long long u0 = blockIdx.x < active ? units * blockIdx.x / active : units;
    const long long u1 = blockIdx.x < active ? units * (blockIdx.x + 1) / active : units;
    if (tid < 2) infos[2 * blockIdx.x + tid] = PieceInfo{-1, 0, 0, 0};
    if (u0 >= u1) return;

    // the block's first unit
    Cursor load;
    {
        int lo = 0, hi = kThreads;  // the last chunk that begins at or before it
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (chunk[mid] <= u0) lo = mid;
            else hi = mid;
        }
        long long rest = u0 - chunk[lo];
        int b = lo * each;
        Span s = span_of<NR>(a, b, group);
        while (rest >= s.units(a.heads)) {
            rest -= s.units(a.heads);
            s = span_of<NR>(a, ++b, group);
        }
        load.b = b;
        load.s = s;
        const int item = static_cast<int>(rest / s.tiles);
        load.head = item / s.row_tiles;
        load.row_tile = item - load.head * s.row_tiles;
        load.tile = static_cast<int>(rest % s.tiles);
    }
    __syncthreads();  // every warp has searched: sm.join is free, also for a warp that has no unit before the first join
    Cursor at = load;  // the block's place: the segment that all its warps are in
    long long left = u1 - u0;
    load.tile += warp;
    settle<NR>(a, load, group);
    long long to_load = left > warp ? (left - warp + kWarps - 1) / kWarps : 0;  // this warp's units

    const int page_size = 1 << a.page_shift;
    const uint32_t ring = ptx::smem_u32(&sm.ring[warp][0][0][0]);
    constexpr int kTile = Smem<DP, NR>::kTile;
    int fill = 0;  // the stage to fill next
    // the table entries of the unit to load next, read one unit ahead
    auto entries = [&](const Cursor& c, int2& p) {
        const int32_t* const row = a.table + c.b * a.stride;
        const int t0 = c.tile * kTok, t1 = t0 + 16;
        p.x = t0 < c.s.r.length ? row[t0 >> a.page_shift] : -1;
        p.y = t1 < c.s.r.length ? row[t1 >> a.page_shift] : -1;
    };
    int2 next = make_int2(-1, -1);
    if (to_load > 0) entries(load, next);
    // fills a stage with the unit under the cursor; the cursor moves on
    auto issue = [&]() {
        if (to_load > 0) {
            int2 p = next;
            // an entry outside the pool hides its tokens: page 0 is loaded, and not looked at
            if (p.x < 0 || p.x >= a.pages) p.x = -1;
            if (p.y < 0 || p.y >= a.pages) p.y = -1;
            const int head = load.head;
            const int t0 = load.tile * kTok;
            if (lane < 4) {
                const int pg = lane < 2 ? p.x : p.y;
                const uint32_t to = ptx::smem_u32(&sm.scale[warp][fill][lane]);
                if (pg >= 0) {
                    const float* const from = (lane & 1 ? a.v_scale : a.k_scale) + static_cast<int64_t>(pg) * a.heads + head;
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(to), "l"(from) : "memory");
                } else {
                    sm.scale[warp][fill][lane] = 0.0f;
                }
            }
            if (lane == 0) {
                sm.page[warp][fill] = p;
                const uint32_t bar = ptx::smem_u32(&sm.full[warp][fill]);
                const uint32_t dst = ring + fill * 2 * kTile;
                if (p.x < 0 && p.y < 0) {
                    ptx::mbar_arrive(bar);  // nothing to load
                } else {
                    ptx::mbar_arrive_expect_tx(bar, 2 * kTile);
                    const int off = head * page_size + (t0 & (page_size - 1));
                    const int px = max(p.x, 0);
                    ptx::tma_load_3d(dst, &maps.k, 0, off, px, bar);
                    ptx::tma_load_3d(dst + kTile, &maps.v, 0, off, px, bar);
                    if (page_size == 16) {
                        const int py = max(p.y, 0);
                        ptx::tma_load_3d(dst + kTile / 2, &maps.k, 0, off, py, bar);
                        ptx::tma_load_3d(dst + kTile + kTile / 2, &maps.v, 0, off, py, bar);
                    }
                }
            }
            fill = fill + 1 == kStages ? 0 : fill + 1;
            --to_load;
            load.tile += kWarps;
            settle<NR>(a, load, group);
            if (to_load > 0) entries(load, next);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");  // one a unit, counted
    };
    for (int s = 0; s < kStages; ++s) issue();

    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    int turn = warp;  // units until this warp's next one
    while (left > 0) {
        // ---- a segment: the rest of this (request, head, row tile), as far as the block's range goes
        const Request r = at.s.r;
        const int head = at.head, row_tile = at.row_tile;
        const int first = at.tile;
        const int count = static_cast<int>(min(static_cast<long long>(at.s.tiles - first), left));
        const int rows_in = min(kRows, r.n * group - row_tile * kRows);

        // q, scaled to fp16's range: the thread's part (a quarter of the dimensions) of rows g, g + 8
        uint32_t qf[NR][KS][2];
        float factor[NR][2];  // of rows 2 q4, 2 q4 + 1 (+ 8)
        int sees[NR][2];      // positions that those see
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            const int row = nr * 8 + g, rr = row_tile * kRows + row;
            const bool live = row < rows_in;
            const int i = live ? rr / group : 0;
            const uint16_t* const src = static_cast<const uint16_t*>(a.q) + (r.row0 + i) * a.q_token_stride +
                                        static_cast<int64_t>(head * group + (live ? rr % group : 0)) * a.q_head_stride +
                                        q4 * (DP / 4);
            uint32_t w[DP / 8];
#pragma unroll
            for (int c = 0; c < DP / 32; ++c) {  // 8 dimensions
                uint4 v = make_uint4(0, 0, 0, 0);
                if (live && q4 * (DP / 4) + c * 8 < a.dim) {
                    if (q_wide) {
                        v = __ldg(reinterpret_cast<const uint4*>(src) + c);
                    } else {
                        const uint16_t* const s = src + c * 8;
                        v.x = s[0] | (static_cast<uint32_t>(s[1]) << 16);
                        v.y = s[2] | (static_cast<uint32_t>(s[3]) << 16);
                        v.z = s[4] | (static_cast<uint32_t>(s[5]) << 16);
                        v.w = s[6] | (static_cast<uint32_t>(s[7]) << 16);
                    }
                }
                w[4 * c] = v.x;
                w[4 * c + 1] = v.y;
                w[4 * c + 2] = v.z;
                w[4 * c + 3] = v.w;
            }
            float most = 0.0f;
#pragma unroll
            for (int c = 0; c < DP / 8; ++c) {
                const float2 f = widen_q(w[c], bf16);
                most = fmaxf(most, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 1));
            most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, 2));
            const int shift = row_shift(most);
            const float2 up = power_of_two(shift), down = power_of_two(-shift);
#pragma unroll
            for (int c = 0; c < DP / 8; ++c) {
                const float2 f = widen_q(w[c], bf16);
                qf[nr][c >> 1][c & 1] = pack_half(f.x * up.x * up.y, f.y * up.x * up.y);
            }
            const float of_row = a.scale * 1.44269504088896341f * down.x * down.y;
            const int row_sees = live ? r.before + i + 1 : 0;
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                factor[nr][e] = __shfl_sync(0xffffffffu, of_row, 4 * (2 * q4 + e));
                sees[nr][e] = __shfl_sync(0xffffffffu, row_sees, 4 * (2 * q4 + e));
            }
        }
        const int all_see = r.before + (row_tile * kRows) / group + 1;  // what even the first row sees

        float o[MB][NR][4];
#pragma unroll
        for (int j = 0; j < MB; ++j)
#pragma unroll
            for (int nr = 0; nr < NR; ++nr) o[j][nr][0] = o[j][nr][1] = o[j][nr][2] = o[j][nr][3] = 0.0f;
        // A row's first reference comes from its first token, whatever its score: until then 0 stands in, and its bit in
        // `have` is clear.  A unit's weights are looked at again where one is above `limit`: in every unit until all rows
        // that see anything have a reference.
        float ref[NR][2], l[NR][2], limit = -INFINITY;
        uint32_t have = 0;
#pragma unroll
        for (int nr = 0; nr < NR; ++nr) {
            ref[nr][0] = ref[nr][1] = 0.0f;
            l[nr][0] = l[nr][1] = 0.0f;
        }
        float c = 0.0f, logc = -127.0f;  // and its log2
        bool some = false;               // whether o holds anything
        auto rescale = [&](const float (&keep)[NR][2]) {
#pragma unroll
            for (int j = 0; j < MB; ++j)
#pragma unroll
                for (int nr = 0; nr < NR; ++nr) {
                    o[j][nr][0] *= keep[nr][0];
                    o[j][nr][1] *= keep[nr][1];
                    o[j][nr][2] *= keep[nr][0];
                    o[j][nr][3] *= keep[nr][1];
                }
        };

        int done = turn;
        for (; done < count; done += kWarps) {
            const int t0 = (first + done) * kTok;
            if (ok) ok = __all_sync(0xffffffffu, ptx::mbar_wait(ptx::smem_u32(&sm.full[warp][stage]), phase, err));
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
            __syncwarp();  // the scales that other lanes fetched
            const int2 page = sm.page[warp][stage];
            const float4 sc = *reinterpret_cast<const float4*>(sm.scale[warp][stage]);
            const float ks[2] = {sc.x, sc.z}, vs[2] = {sc.y, sc.w};
            const uint32_t kt = ring + stage * 2 * kTile, vt = kt + kTile;
            // every row sees every token
            const bool whole = t0 + kTok <= all_see && page.x >= 0 && page.y >= 0;

            float s[2][NR][4];
#pragma unroll
            for (int mb = 0; mb < 2; ++mb) {
#pragma unroll
                for (int nr = 0; nr < NR; ++nr) s[mb][nr][0] = s[mb][nr][1] = s[mb][nr][2] = s[mb][nr][3] = 0.0f;
                uint32_t w[2][KS];  // codes of tokens g, g + 8
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int c = 0; c < DP / 64; ++c) {
                        const uint4 v = lds16(kt + chunk_at<DP>(mb * 16 + h * 8 + g, q4 * (DP / 64) + c));
                        w[h][4 * c] = v.x;
                        w[h][4 * c + 1] = v.y;
                        w[h][4 * c + 2] = v.z;
                        w[h][4 * c + 3] = v.w;
                    }
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const uint32_t a0 = widen_low(w[0][k]), a1 = widen_low(w[1][k]);
                    const uint32_t a2 = widen_high(w[0][k]), a3 = widen_high(w[1][k]);
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr) mma16816(s[mb][nr], a0, a1, a2, a3, qf[nr][k][0], qf[nr][k][1]);
                }
            }
            // ---- softmax weights: rows 2 q4, 2 q4 + 1 (+ 8), tokens g, g + 8 of each 16
            float vmost = vs[0] <= 3.402823466e38f ? fmaxf(vs[0], 0.0f) : 0.0f;
            vmost = vs[1] <= 3.402823466e38f ? fmaxf(vmost, vs[1]) : vmost;
            if (vmost > c) {  // the same in every lane
                const float to = __int_as_float(min((__float_as_int(vmost) & 0x7f800000) + (1 << 23), 0x7f000000));
                if (some) {
                    float keep[NR][2];
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr) keep[nr][0] = keep[nr][1] = c / to;
                    rescale(keep);
                }
                c = to;
                logc = static_cast<float>((__float_as_int(to) >> 23) - 127);
            }
            some = true;
            // log2 of the weights' factors; 2^-60 of c stands in for smaller scales (their fp16 weights are 0 then)
            // and for one that is not finite, whose weights become NaN below: the sums do not depend on it
            float lw[2], out_of[2];
            const bool broken = !(vs[0] <= 3.402823466e38f && vs[1] <= 3.402823466e38f);
#pragma unroll
            for (int mb = 0; mb < 2; ++mb) {
                const bool usual = vs[mb] > c * 8.67361738e-19f && vs[mb] <= 3.402823466e38f;
                lw[mb] = usual ? __log2f(vs[mb]) + (kLogStart - logc) : kLogStart - 60.0f;
                out_of[mb] = exp2_fast(-lw[mb]);
            }
            float z[2][NR][4];  // log2 of the weights
            auto weigh = [&]() {
                float top = -INFINITY;
#pragma unroll
                for (int mb = 0; mb < 2; ++mb)
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int e = i & 1;
                            float x = fmaf(s[mb][nr][i], factor[nr][e] * ks[mb], lw[mb] - ref[nr][e]);
                            if (!whole) {
                                const int pos = t0 + mb * 16 + (i >> 1) * 8 + g;
                                x = pos < sees[nr][e] && (mb ? page.y : page.x) >= 0 ? x : -INFINITY;
                            }
                            z[mb][nr][i] = x;
                            top = fmaxf(top, x);
                        }
                return top;
            };
            // (Written as a loop, the weights' code is there once: 2% of a batch of single tokens.)
            float most = limit;
#pragma unroll 1
            for (int turn = 0; __any_sync(0xffffffffu, weigh() > most) && turn < 2; ++turn) {
                float keep[NR][2];
                bool all = true;
                most = kLogTop;
#pragma unroll
                for (int nr = 0; nr < NR; ++nr)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = fmaxf(fmaxf(z[0][nr][e], z[0][nr][2 + e]), fmaxf(z[1][nr][e], z[1][nr][2 + e]));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 4));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 8));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
                        keep[nr][e] = 1.0f;
                        const uint32_t bit = 1u << (2 * nr + e);
                        if (top > (have & bit ? kLogTop : -INFINITY)) {
                            const float to = ref[nr][e] + (ceilf(top) - kLogStart);
                            keep[nr][e] = have & bit ? exp2_fast(ref[nr][e] - to) : 0.0f;
                            ref[nr][e] = to;
                            l[nr][e] *= keep[nr][e];
                            have |= bit;
                        }
                        all = all && ((have & bit) || sees[nr][e] <= 0);
                    }
                limit = __all_sync(0xffffffffu, all) ? kLogTop : -INFINITY;
                rescale(keep);
            }
            uint32_t pf[2][NR][2], pl[2][NR][2];  // B fragments of the two 16-token steps; what their rounding left
#pragma unroll
            for (int mb = 0; mb < 2; ++mb)
#pragma unroll
                for (int nr = 0; nr < NR; ++nr) {
                    float p[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) p[i] = exp2_fast(z[mb][nr][i]);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        l[nr][e] = fmaf(p[e] + p[2 + e], out_of[mb], l[nr][e]);
                    }
                    if (broken) {
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if (!(vs[mb] <= 3.402823466e38f) && z[mb][nr][i] != -INFINITY) p[i] = __int_as_float(0x7fffffff);
                    }
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t h = pack_half(p[2 * i], p[2 * i + 1]);
                        pf[mb][nr][i] = transpose8(h);
                        if (kFine) pl[mb][nr][i] = transpose8(left_of(h, p[2 * i], p[2 * i + 1]));
                    }
                }
            // ---- values
            bool odd = false;  // a NaN code that some row may not see
#pragma unroll
            for (int st = 0; st < 2; ++st) {
                uint32_t v[4][VW];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int row = st * 16 + q4 * 2 + (i & 1) + (i >> 1) * 8;
                    if (DP == 128) {
                        const uint4 x = lds16(vt + chunk_at<DP>(row, g));
                        v[i][0] = x.x;
                        v[i][1] = x.y;
                        v[i][VW - 2] = x.z;
                        v[i][VW - 1] = x.w;
                    } else {
                        const uint2 x = lds8(vt + chunk_at<DP>(row, g >> 1) + (g & 1) * 8);
                        v[i][0] = x.x;
                        v[i][1] = x.y;
                    }
                    if (!whole) {
                        // no row's token: its codes may be anything; a token that some rows
                        // see: its NaN codes are set apart
                        const bool live = t0 + row < r.length && (st ? page.y : page.x) >= 0;
#pragma unroll
                        for (int k = 0; k < VW; ++k) {
                            const uint32_t nan = __vcmpeq4(v[i][k] & 0x7f7f7f7fu, 0x7f7f7f7fu);
                            odd = odd || (live && nan != 0);
                            v[i][k] = live ? v[i][k] & ~nan : 0u;
                        }
                    }
                }
#pragma unroll
                for (int k = 0; k < VW; ++k) {
                    const uint32_t x01 = __byte_perm(v[0][k], v[1][k], 0x5140), x23 = __byte_perm(v[0][k], v[1][k], 0x7362);
                    const uint32_t y01 = __byte_perm(v[2][k], v[3][k], 0x5140), y23 = __byte_perm(v[2][k], v[3][k], 0x7362);
                    const uint32_t a0 = widen_low(x01), a1 = widen_high(x01), a2 = widen_low(y01), a3 = widen_high(y01);
                    const uint32_t b0 = widen_low(x23), b1 = widen_high(x23), b2 = widen_low(y23), b3 = widen_high(y23);
#pragma unroll
                    for (int nr = 0; nr < NR; ++nr) {
                        mma16816(o[2 * k][nr], a0, a1, a2, a3, pf[st][nr][0], pf[st][nr][1]);
                        mma16816(o[2 * k + 1][nr], b0, b1, b2, b3, pf[st][nr][0], pf[st][nr][1]);
                        if (kFine) {
                            mma16816(o[2 * k][nr], a0, a1, a2, a3, pl[st][nr][0], pl[st][nr][1]);
                            mma16816(o[2 * k + 1][nr], b0, b1, b2, b3, pl[st][nr][0], pl[st][nr][1]);
                        }
                    }
                }
            }
            if (!whole && __any_sync(0xffffffffu, odd)) {
                // the rows that see a NaN code get it, the others do not
#pragma unroll 1
                for (int row = 0; row < kTok; ++row) {
                    const int pos = t0 + row;
                    if (pos >= r.length || (row < 16 ? page.x : page.y) < 0) continue;
#pragma unroll
                    for (int j = 0; j < MB; ++j) {
                        // m-block j: the thread's dimensions g * DP / 8 + 2 j, + 1
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int d = g * (DP / 8) + 2 * j + e;
                            uint32_t code;
                            asm volatile("ld.shared.u8 %0, [%1];" : "=r"(code) : "r"(vt + chunk_at<DP>(row, d >> 4) + (d & 15)));
                            if ((code & 0x7f) == 0x7f) {
#pragma unroll
                                for (int nr = 0; nr < NR; ++nr) {
                                    if (pos < sees[nr][0]) o[j][nr][2 * e] = __int_as_float(0x7fffffff);
                                    if (pos < sees[nr][1]) o[j][nr][2 * e + 1] = __int_as_float(0x7fffffff);
                                }
                            }
                        }
                    }
                }
            }
            __syncwarp();  // every lane is done with the stage
            issue();
            if (++stage == kStages) {
                stage = 0;
                phase ^= 1;
            }
        }
        turn = done - count;  // into the next segment

        // ---- the segment's end: the warps' sums are joined, 4 vectors of every lane at a time, each by one warp
#pragma unroll
        for (int nr = 0; nr < NR; ++nr)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                l[nr][e] += __shfl_xor_sync(0xffffffffu, l[nr][e], 4);
                l[nr][e] += __shfl_xor_sync(0xffffffffu, l[nr][e], 8);
                l[nr][e] += __shfl_xor_sync(0xffffffffu, l[nr][e], 16);
                if (g == 0) {
                    sm.m[warp][nr * 8 + 2 * q4 + e] = l[nr][e] == 0.0f ? kNothing : ref[nr][e];
                    sm.l[warp][nr * 8 + 2 * q4 + e] = l[nr][e];
                }
            }
        if (lane == 0) sm.c[warp] = c * 0.0078125f;  // 2^-7 c: what a weight of 1 stands for
        const bool begins = first == 0, ends = first + count == at.s.tiles;
        const bool cut = !(begins && ends);
        const int slot = 2 * blockIdx.x + (begins ? 1 : 0);
#pragma unroll
        for (int k0 = 0; k0 < kVectors; k0 += 4) {
            if (k0) __syncthreads();
#pragma unroll
            for (int k = k0; k < k0 + 4; ++k) {
                const int e = k / VR, i = k % VR, nr = e >> 1, b = e & 1;
                sm.join[warp][k - k0][lane] =
                    make_float4(o[2 * i][nr][b], o[2 * i][nr][2 + b], o[2 * i + 1][nr][b], o[2 * i + 1][nr][2 + b]);
            }
            __syncthreads();
            if (warp < 4) {
                const int k = k0 + warp;
                int row, dim;
                vector_place<DP>(k, lane, row, dim);
                float big = kNothing, sum = 0.0f;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) big = fmaxf(big, sm.m[w][row]);
                float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
                for (int w = 0; w < kWarps; ++w) {
                    const float lw = sm.l[w][row];
                    if (lw == 0.0f) continue;  // a warp that saw nothing has no part, NaN sums stay
                    const float f = exp2_fast(sm.m[w][row] - big), fc = f * sm.c[w];
                    const float4 y = sm.join[w][warp][lane];
                    sum = fmaf(lw, f, sum);
                    x.x = fmaf(y.x, fc, x.x);
                    x.y = fmaf(y.y, fc, x.y);
                    x.z = fmaf(y.z, fc, x.z);
                    x.w = fmaf(y.w, fc, x.w);
                }
                if (cut) {
                    pieces[slot].o[k * 32 + lane] = x;
                    if (dim == 0) {
                        pieces[slot].m[row] = big;
                        pieces[slot].l[row] = sum;
                    }
                } else {
                    write_vector<DP, NR>(a, r, head, row_tile, group, k, lane, x, sum, big, out_wide);
                }
            }
        }
        if (cut && tid == 0) infos[slot] = PieceInfo{at.b, head * at.s.row_tiles + row_tile, begins, ends};
        __syncthreads();  // sm.join, sm.m and sm.l are free again
        left -= count;
        at.tile += count;
        if (left > 0) settle<NR>(a, at, group);
    }
}

// One block for each block of the first launch: if a request was cut behind
// its first tokens there, the block joins all of its pieces, in order.
template <int DP, int NR>
__global__ void __launch_bounds__(256) attention_join_kernel(const AttentionArgs a, int blocks, const PieceInfo* infos,
                                                             const Piece<DP, NR>* pieces, bool out_wide) {
    constexpr int kRows = 8 * NR, kMost = 64;  // pieces whose factors are kept at a time
    __shared__ float factor[kMost][kRows], sum[kMost][kRows];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const PieceInfo info = infos[2 * blockIdx.x + 1];
    if (info.request < 0 || info.ends) return;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int group = a.q_heads / a.heads;
    const Span s = span_of<NR>(a, info.request, group);
    const int head = info.unit / s.row_tiles, row_tile = info.unit - head * s.row_tiles;
    const int first = blockIdx.x;
    int n = 1;  // pieces: of this block and the blocks behind it
    while (first + n < blocks) {
        const int c = first + n + lane;
        const unsigned ends = __ballot_sync(0xffffffffu, c >= blocks || infos[2 * c].ends);
        n += ends ? __ffs(ends) : 32;
        if (ends) break;
    }
    n = min(n, blocks - first);
    auto piece = [&](int i) { return pieces + 2 * (first + i) + (i == 0 ? 1 : 0); };
    constexpr int V = 2 * NR * DP / 32, kEach = (V + 7) / 8;
    float m[kEach], l[kEach];
    float4 x[kEach];
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        m[j] = kNothing;
        l[j] = 0.0f;
        x[j] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    for (int i0 = 0; i0 < n; i0 += kMost) {
        const int some = min(kMost, n - i0);
        for (int i = tid; i < some * kRows; i += 256) {
            factor[i / kRows][i % kRows] = piece(i0 + i / kRows)->m[i % kRows];
            sum[i / kRows][i % kRows] = piece(i0 + i / kRows)->l[i % kRows];
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
            const int k = warp + 8 * j;
            if (k >= V) continue;
            int row, dim;
            vector_place<DP>(k, lane, row, dim);
            float big = m[j];
            for (int i = 0; i < some; ++i) big = fmaxf(big, factor[i][row]);
            const float keep = exp2_fast(m[j] - big);
            m[j] = big;
            l[j] *= keep;
            x[j].x *= keep;
            x[j].y *= keep;
            x[j].z *= keep;
            x[j].w *= keep;
#pragma unroll 8
            for (int i = 0; i < some; ++i) {
                const float4 y = piece(i0 + i)->o[k * 32 + lane];
                const float li = sum[i][row], f = li == 0.0f ? 0.0f : exp2_fast(factor[i][row] - big);
                // a piece that saw nothing holds zeros
                l[j] = fmaf(li, f, l[j]);
                x[j].x = fmaf(y.x, f, x[j].x);
                x[j].y = fmaf(y.y, f, x[j].y);
                x[j].z = fmaf(y.z, f, x[j].z);
                x[j].w = fmaf(y.w, f, x[j].w);
            }
        }
        __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < kEach; ++j) {
        const int k = warp + 8 * j;
        if (k < V) write_vector<DP, NR>(a, s.r, head, row_tile, group, k, lane, x[j], l[j], m[j], out_wide);
    }
}

bool wide_rows(const void* p, int64_t token, int64_t head, int64_t bytes) {
    return ((reinterpret_cast<uintptr_t>(p) | static_cast<uintptr_t>(token * 2) | static_cast<uintptr_t>(head * 2)) &
            (bytes - 1)) == 0;
}

size_t round16(size_t n) { return (n + 15) & ~static_cast<size_t>(15); }

template <int DP, int NR, bool kFine>
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
    const uint32_t box[3] = {DP, page < kTok ? page : kTok, 1};
    // a cache without pages: nothing is loaded, but a map needs an address
    const void* const k = a.pages > 0 ? a.k_cache : a.workspace;
    const void* const v = a.pages > 0 ? a.v_cache : a.workspace;
    if (!encode_tmap_bytes(&maps.k, k, dims, strides, box) || !encode_tmap_bytes(&maps.v, v, dims, strides, box))
        return cudaErrorInvalidValue;
    uint8_t* const w = static_cast<uint8_t*>(a.workspace);
    PieceInfo* const infos = reinterpret_cast<PieceInfo*>(w);
    Piece<DP, NR>* const pieces = reinterpret_cast<Piece<DP, NR>*>(w + round16(sizeof(PieceInfo) * 2 * blocks));
    const size_t smem = sizeof(Smem<DP, NR>) + 1024;
    static std::atomic<uint64_t> allowed{0};
    e = allow_shared(attention_split_kernel<DP, NR, kFine>, smem, dev, allowed);
    if (e != cudaSuccess) return e;
    const bool q_wide = wide_rows(a.q, a.q_token_stride, a.q_head_stride, 16);
    const bool out_wide = wide_rows(a.out, a.out_token_stride, a.out_head_stride, 8);
    attention_split_kernel<DP, NR, kFine><<<blocks, 32 * Shape<NR>::kWarps, smem, stream>>>(
        a, maps, device_error_word(), infos, pieces, q_wide, out_wide);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(256);
    cfg.stream = stream;
    cudaLaunchAttribute attr;
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, attention_join_kernel<DP, NR>, a, blocks, static_cast<const PieceInfo*>(infos),
                              static_cast<const Piece<DP, NR>*>(pieces), out_wide);
}

template <int NR>
cudaError_t launch_rows(const AttentionArgs& a, cudaStream_t stream) {
    if (a.dtype == kBF16) return a.dim <= 64 ? launch<64, NR, false>(a, stream) : launch<128, NR, false>(a, stream);
    return a.dim <= 64 ? launch<64, NR, true>(a, stream) : launch<128, NR, true>(a, stream);
}

}  // namespace

size_t attention_split_workspace(int64_t dim, int sms) {
    const size_t piece = dim <= 64 ? sizeof(Piece<64, 2>) : sizeof(Piece<128, 2>);
    return round16(sizeof(PieceInfo) * 2 * sms) + 2 * piece * sms;
}

cudaError_t launch_attention_split(const AttentionArgs& a, cudaStream_t stream) {
    // One block of 8 rows, or two, whose registers leave room for fewer warps.  64 requests of 4700 tokens, bf16: 8 rows
    // 132 us with one and 179 with two, 12 rows 222 (the cache read twice) and 185.
    const bool one = a.max_added * (a.q_heads / a.heads) <= 8;
    return one ? launch_rows<1>(a, stream) : launch_rows<2>(a, stream);
}

}  // namespace lik
