// api_serve.cu -- C entry points of a serving step over a cache in 8 bits
// (include/lik.h): argument checks and launches.
#include "lik.h"
#include "lik_internal.h"
#include "serve.h"
#include "validate.h"

namespace lik {
namespace {

typedef long long ll;

constexpr int64_t kMaxElems = int64_t(1) << 48;  // no buffer is as large; keeps offsets far inside 64 bits

lik_status check_page_size(int64_t page_size, int* shift) {
    for (int s = 4; s <= 8; ++s) {
        if (page_size == int64_t(1) << s) {
            *shift = s;
            return LIK_OK;
        }
    }
    return fail(LIK_ERR_UNSUPPORTED, "page_size must be 16, 32, 64, 128 or 256 (got %lld)", static_cast<ll>(page_size));
}

lik_status check_requests(int64_t requests) {
    if (requests < 0) return fail(LIK_ERR_INVALID_ARG, "negative size");
    if (requests > kMaxRequests)
        return fail(LIK_ERR_UNSUPPORTED, "requests %lld > %d", static_cast<ll>(requests), kMaxRequests);
    return LIK_OK;
}

lik_status check_table(int64_t requests, int64_t cols, int64_t stride) {
    if (cols < 0) return fail(LIK_ERR_INVALID_ARG, "negative size");
    if (cols > INT32_MAX) return fail(LIK_ERR_UNSUPPORTED, "table_cols %lld > 2^31 - 1", static_cast<ll>(cols));
    if (stride < cols && requests > 1)
        return fail(LIK_ERR_INVALID_ARG, "table_stride %lld < table_cols %lld", static_cast<ll>(stride),
                    static_cast<ll>(cols));
    if (stride > (int64_t(1) << 31))
        return fail(LIK_ERR_UNSUPPORTED, "table_stride %lld > 2^31", static_cast<ll>(stride));
    return LIK_OK;
}

// rows x heads x dim with heads and dim of a cache
lik_status check_rows(int64_t rows, int64_t heads, int64_t dim) {
    if (rows < 0 || heads < 0) return fail(LIK_ERR_INVALID_ARG, "negative size");
    if (heads < 1 || heads > 1024)
        return fail(LIK_ERR_UNSUPPORTED, "heads must lie in [1, 1024] (got %lld)", static_cast<ll>(heads));
    if (dim < 16 || dim > kMaxHeadDim || dim % 16)
        return fail(LIK_ERR_UNSUPPORTED, "dim must be a multiple of 16 in [16, %d] (got %lld)", kMaxHeadDim,
                    static_cast<ll>(dim));
    return LIK_OK;
}

// Strides of a [rows, heads, dim] tensor: not negative, and its extent bounded.
lik_status check_strides(int64_t rows, int64_t heads, int64_t token, int64_t head, const char* name) {
    if (token < 0 || head < 0) return fail(LIK_ERR_INVALID_ARG, "%s has a negative stride", name);
    if (token > (int64_t(1) << 32) || head > (int64_t(1) << 32) || (rows > 0 && rows * token > kMaxElems))
        return fail(LIK_ERR_UNSUPPORTED, "%s spans more than 2^48 elements", name);
    return LIK_OK;
}

// An output whose rows of dim elements do not overlap: heads inside tokens or tokens inside heads, whichever are
// further apart (a single one may have any stride).
lik_status check_spread(int64_t rows, int64_t heads, int64_t dim, int64_t token, int64_t head, const char* name) {
    if (rows == 0) return LIK_OK;
    const bool one_row = rows <= 1, one_head = heads <= 1;
    const bool inside = (one_head || head >= dim) && (one_row || token >= (one_head ? 0 : (heads - 1) * head) + dim);
    const bool across = (one_row || token >= dim) && (one_head || head >= (one_row ? 0 : (rows - 1) * token) + dim);
    if (inside || across) return LIK_OK;
    return fail(LIK_ERR_INVALID_ARG, "%s has rows that overlap (strides %lld and %lld)", name, static_cast<ll>(token),
                static_cast<ll>(head));
}

int64_t span(int64_t rows, int64_t token, int64_t heads, int64_t head, int64_t dim) {
    return rows > 0 && heads > 0 ? (rows - 1) * token + (heads - 1) * head + dim : 0;
}

lik_status check_pool(int64_t pages, int64_t heads, int64_t page_size, int64_t dim) {
    if (pages < 0) return fail(LIK_ERR_INVALID_ARG, "negative size");
    if (pages > INT32_MAX) return fail(LIK_ERR_UNSUPPORTED, "pages %lld > 2^31 - 1", static_cast<ll>(pages));
    if (pages * heads > kMaxElems / (page_size * dim))
        return fail(LIK_ERR_UNSUPPORTED, "the cache has more than 2^48 codes");
    return LIK_OK;
}

struct Bytes {
    const char* name;
    const void* ptr;
    int64_t bytes;
};

// An output that overlaps any of the others is refused.
lik_status check_apart(const Bytes* outs, int n_out, const Bytes* ins, int n_in) {
    for (int i = 0; i < n_out; ++i) {
        const uintptr_t o0 = reinterpret_cast<uintptr_t>(outs[i].ptr), o1 = o0 + outs[i].bytes;
        if (!outs[i].ptr || outs[i].bytes <= 0) continue;
        for (int j = 0; j < n_in + n_out; ++j) {
            const Bytes& x = j < n_in ? ins[j] : outs[j - n_in];
            if (j - n_in == i || !x.ptr || x.bytes <= 0) continue;
            const uintptr_t x0 = reinterpret_cast<uintptr_t>(x.ptr), x1 = x0 + x.bytes;
            if (o0 < x1 && x0 < o1) return fail(LIK_ERR_INVALID_ARG, "%s overlaps %s", outs[i].name, x.name);
        }
    }
    return LIK_OK;
}

lik_status check_workspace(const void* p, size_t bytes, size_t need, int dev) {
    if (!p || bytes < need)
        return fail(LIK_ERR_INVALID_ARG, "workspace of %zu bytes given, this call needs %zu", p ? bytes : 0, need);
    lik_status st = check_pointer(p, dev, "workspace");
    if (st == LIK_OK) st = check_aligned(p, 16, "workspace");
    return st;
}

lik_status check_scale(float scale) {
    if (!(scale >= 1e-30f && scale <= 1e30f))
        return fail(LIK_ERR_INVALID_ARG, "scale must lie in [1e-30, 1e30] (got %g)", static_cast<double>(scale));
    return LIK_OK;
}

size_t elem_bytes(lik_dtype t) { return t == LIK_F32 ? 4 : 2; }

lik_status check_attention(int64_t rows, int64_t q_heads, int64_t heads, int64_t dim, int64_t requests,
                           int64_t page_size, int64_t table_cols, int64_t max_added, int* shift) {
    lik_status st = check_page_size(page_size, shift);
    if (st == LIK_OK) st = check_rows(rows, heads, dim);
    if (st == LIK_OK) st = check_requests(requests);
    if (st != LIK_OK) return st;
    if (q_heads < 1 || q_heads % heads || q_heads / heads > 128)
        return fail(LIK_ERR_UNSUPPORTED, "q_heads %lld must be 1 to 128 times heads %lld", static_cast<ll>(q_heads),
                    static_cast<ll>(heads));
    // the kernels count a request's rows of all heads, rounded up to an item, in 32 bits
    if (rows > INT32_MAX || rows * q_heads > (int64_t(1) << 30))
        return fail(LIK_ERR_UNSUPPORTED, "rows * q_heads > 2^30");
    if (table_cols < 0 || max_added < 0) return fail(LIK_ERR_INVALID_ARG, "negative size");
    // positions are counted in 32 bits, and looked up to 16 tiles of 64 tokens ahead
    if (table_cols * page_size > INT32_MAX - 4095)
        return fail(LIK_ERR_UNSUPPORTED, "a table row of more than 2^31 - 4096 tokens");
    return LIK_OK;
}

}  // namespace
}  // namespace lik

using namespace lik;

// fit: whether most and missing are wanted too
static lik_status cache_slots(const int32_t* cached, const int32_t* added, const int32_t* held, int64_t requests,
                              int64_t page_size, const int32_t* free_pages, int64_t free_capacity,
                              const int32_t* free_count, int32_t* block_table, int64_t table_cols,
                              int64_t table_stride, int32_t* held_out, int32_t* lengths, int32_t* offsets,
                              int64_t* slots, int64_t slot_capacity, int32_t* free_left, bool fit, int32_t* most,
                              int32_t* missing, cudaStream_t stream) {
    clear_message();
    SlotsArgs a{};
    lik_status st = check_page_size(page_size, &a.page_shift);
    if (st == LIK_OK) st = check_requests(requests);
    if (st == LIK_OK) st = check_table(requests, table_cols, table_stride);
    if (st != LIK_OK) return st;
    if (free_capacity < 0 || slot_capacity < 0) return fail(LIK_ERR_INVALID_ARG, "negative size");
    if (free_capacity > INT32_MAX || slot_capacity > INT32_MAX)
        return fail(LIK_ERR_UNSUPPORTED, "free_capacity or slot_capacity > 2^31 - 1");
    int dev = 0;
    if ((st = check_device(&dev)) != LIK_OK) return st;
    const int64_t B = requests, span_table = B > 0 ? (B - 1) * table_stride + table_cols : 0;
    const Spec specs[] = {
        {"cached", cached, true, B},
        {"added", added, true, B},
        {"held", held, true, B},
        {"free_pages", free_pages, true, free_capacity},
        {"free_count", free_count, true, 1},
        {"block_table", block_table, true, table_cols > 0 ? span_table : 0},
        {"held_out", held_out, true, B},
        {"lengths", lengths, true, B},
        {"offsets", offsets, true, B + 1},
        {"free_left", free_left, true, 1},
        {"slots", slots, true, slot_capacity},
        {"most", most, fit, B},
        {"missing", missing, fit, 1},
    };
    if ((st = check_buffers(dev, specs, fit ? 13 : 11)) != LIK_OK) return st;
    for (const Spec& s : specs)
        if ((st = check_aligned(s.ptr, s.ptr == slots ? 8 : 4, s.name)) != LIK_OK) return st;
    const Bytes ins[] = {{"cached", cached, 4 * B},         {"added", added, 4 * B},
                         {"held", held, 4 * B},             {"free_pages", free_pages, 4 * free_capacity},
                         {"free_count", free_count, 4}};
    const Bytes outs[] = {{"block_table", block_table, 4 * specs[5].elems}, {"held_out", held_out, 4 * B},
                          {"lengths", lengths, 4 * B},                      {"offsets", offsets, 4 * (B + 1)},
                          {"slots", slots, 8 * slot_capacity},              {"free_left", free_left, 4},
                          {"most", most, 4 * B},                            {"missing", missing, 4}};
    if ((st = check_apart(outs, 8, ins, 5)) != LIK_OK) return st;
    a.cached = cached;
    a.added = added;
    a.held = held;
    a.requests = static_cast<int>(B);
    a.free_pages = free_pages;
    a.free_capacity = free_capacity;
    a.free_count = free_count;
    a.table = block_table;
    a.cols = table_cols;
    a.stride = table_stride;
    a.held_out = held_out;
    a.lengths = lengths;
    a.offsets = offsets;
    a.slots = slots;
    a.capacity = slot_capacity;
    a.free_left = free_left;
    a.most = most;
    a.missing = missing;
    const cudaError_t e = launch_cache_slots(a, stream);
    return e == cudaSuccess ? LIK_OK : cuda_fail(e, "slot map launch");
}

extern "C" lik_status lik_cache_slots(const int32_t* cached, const int32_t* added, const int32_t* held,
                                      int64_t requests, int64_t page_size, const int32_t* free_pages,
                                      int64_t free_capacity, const int32_t* free_count, int32_t* block_table,
                                      int64_t table_cols, int64_t table_stride, int32_t* held_out, int32_t* lengths,
                                      int32_t* offsets, int64_t* slots, int64_t slot_capacity, int32_t* free_left,
                                      cudaStream_t stream) {
    return cache_slots(cached, added, held, requests, page_size, free_pages, free_capacity, free_count, block_table,
                       table_cols, table_stride, held_out, lengths, offsets, slots, slot_capacity, free_left, false,
                       nullptr, nullptr, stream);
}

extern "C" lik_status lik_cache_slots_fit(const int32_t* cached, const int32_t* added, const int32_t* held,
                                          int64_t requests, int64_t page_size, const int32_t* free_pages,
                                          int64_t free_capacity, const int32_t* free_count, int32_t* block_table,
                                          int64_t table_cols, int64_t table_stride, int32_t* held_out,
                                          int32_t* lengths, int32_t* offsets, int64_t* slots, int64_t slot_capacity,
                                          int32_t* free_left, int32_t* most, int32_t* missing, cudaStream_t stream) {
    return cache_slots(cached, added, held, requests, page_size, free_pages, free_capacity, free_count, block_table,
                       table_cols, table_stride, held_out, lengths, offsets, slots, slot_capacity, free_left, true,
                       most, missing, stream);
}

extern "C" lik_status lik_cache_write(const void* k, const void* v, lik_dtype dtype, int64_t rows, int64_t heads,
                                      int64_t dim, int64_t k_token_stride, int64_t k_head_stride,
                                      int64_t v_token_stride, int64_t v_head_stride, const int64_t* slots,
                                      void* k_cache, void* v_cache, float* k_scale, float* v_scale, int64_t pages,
                                      int64_t page_size, cudaStream_t stream) {
    clear_message();
    WriteArgs a{};
    if (!known_dtype(dtype)) return fail(LIK_ERR_INVALID_ARG, "unknown dtype %d", static_cast<int>(dtype));
    lik_status st = check_page_size(page_size, &a.page_shift);
    if (st == LIK_OK) st = check_rows(rows, heads, dim);
    if (st == LIK_OK && rows > INT32_MAX) st = fail(LIK_ERR_UNSUPPORTED, "rows %lld > 2^31 - 1", static_cast<ll>(rows));
    if (st == LIK_OK) st = check_pool(pages, heads, page_size, dim);
    if (st == LIK_OK) st = check_strides(rows, heads, k_token_stride, k_head_stride, "k");
    if (st == LIK_OK) st = check_strides(rows, heads, v_token_stride, v_head_stride, "v");
    if (st != LIK_OK) return st;
    int dev = 0;
    if ((st = check_device(&dev)) != LIK_OK) return st;
    const int64_t codes = pages * heads * page_size * dim, es = static_cast<int64_t>(elem_bytes(dtype));
    const int64_t k_span = span(rows, k_token_stride, heads, k_head_stride, dim);
    const int64_t v_span = span(rows, v_token_stride, heads, v_head_stride, dim);
    const Spec specs[] = {
        {"k", k, true, k_span},           {"v", v, true, v_span},
        {"slots", slots, true, rows},     {"k_cache", k_cache, true, rows > 0 ? codes : 0},
        {"v_cache", v_cache, true, rows > 0 ? codes : 0},
        {"k_scale", k_scale, true, rows > 0 ? pages * heads : 0},
        {"v_scale", v_scale, true, rows > 0 ? pages * heads : 0},
    };
    if ((st = check_buffers(dev, specs, 7)) != LIK_OK) return st;
    if ((st = check_aligned(k, es, "k")) != LIK_OK || (st = check_aligned(v, es, "v")) != LIK_OK) return st;
    if ((st = check_aligned(slots, 8, "slots")) != LIK_OK) return st;
    if ((st = check_aligned(k_cache, 16, "k_cache")) != LIK_OK || (st = check_aligned(v_cache, 16, "v_cache")) != LIK_OK)
        return st;
    if ((st = check_aligned(k_scale, 4, "k_scale")) != LIK_OK || (st = check_aligned(v_scale, 4, "v_scale")) != LIK_OK)
        return st;
    if (rows == 0 || pages == 0) return LIK_OK;
    const Bytes ins[] = {{"k", k, k_span * es}, {"v", v, v_span * es}, {"slots", slots, 8 * rows}};
    const Bytes outs[] = {{"k_cache", k_cache, codes},
                          {"v_cache", v_cache, codes},
                          {"k_scale", k_scale, 4 * pages * heads},
                          {"v_scale", v_scale, 4 * pages * heads}};
    if ((st = check_apart(outs, 4, ins, 3)) != LIK_OK) return st;
    a.x[0] = k;
    a.x[1] = v;
    a.dtype = static_cast<int>(dtype);
    a.rows = rows;
    a.heads = static_cast<int>(heads);
    a.dim = static_cast<int>(dim);
    a.token_stride[0] = k_token_stride;
    a.token_stride[1] = v_token_stride;
    a.head_stride[0] = k_head_stride;
    a.head_stride[1] = v_head_stride;
    a.slots = slots;
    a.cache[0] = static_cast<uint8_t*>(k_cache);
    a.cache[1] = static_cast<uint8_t*>(v_cache);
    a.scale[0] = k_scale;
    a.scale[1] = v_scale;
    a.pages = pages;
    const cudaError_t e = launch_cache_write(a, stream);
    return e == cudaSuccess ? LIK_OK : cuda_fail(e, "cache write launch");
}

extern "C" lik_status lik_cache_attention_workspace_bytes(int64_t rows, int64_t q_heads, int64_t heads, int64_t dim,
                                                          int64_t requests, int64_t page_size, int64_t table_cols,
                                                          int64_t max_added, size_t* bytes) {
    clear_message();
    if (!bytes) return fail(LIK_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    int shift = 0;
    lik_status st = check_attention(rows, q_heads, heads, dim, requests, page_size, table_cols, max_added, &shift);
    if (st != LIK_OK || rows == 0 || requests == 0) return st;
    int dev = 0;
    if ((st = check_device(&dev)) != LIK_OK) return st;
    *bytes = cache_attention_workspace(rows, q_heads, heads, dim, requests, max_added);
    return LIK_OK;
}

extern "C" lik_status lik_cache_attention(const void* q, lik_dtype dtype, int64_t rows, int64_t q_heads, int64_t dim,
                                          int64_t q_token_stride, int64_t q_head_stride, const void* k_cache,
                                          const void* v_cache, const float* k_scale, const float* v_scale,
                                          int64_t pages, int64_t heads, int64_t page_size, const int32_t* block_table,
                                          int64_t table_cols, int64_t table_stride, const int32_t* offsets,
                                          const int32_t* lengths, int64_t requests, int64_t max_added, float scale,
                                          void* out, int64_t out_token_stride, int64_t out_head_stride, float* lse,
                                          void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    clear_message();
    AttentionArgs a{};
    if (dtype != LIK_F16 && dtype != LIK_BF16) {
        if (dtype == LIK_F32) return fail(LIK_ERR_UNSUPPORTED, "q must be fp16 or bf16");
        return fail(LIK_ERR_INVALID_ARG, "unknown dtype %d", static_cast<int>(dtype));
    }
    lik_status st = check_attention(rows, q_heads, heads, dim, requests, page_size, table_cols, max_added, &a.page_shift);
    if (st == LIK_OK) st = check_pool(pages, heads, page_size, dim);
    if (st == LIK_OK) st = check_table(requests, table_cols, table_stride);
    if (st == LIK_OK) st = check_strides(rows, q_heads, q_token_stride, q_head_stride, "q");
    if (st == LIK_OK) st = check_strides(rows, q_heads, out_token_stride, out_head_stride, "out");
    if (st == LIK_OK) st = check_spread(rows, q_heads, dim, out_token_stride, out_head_stride, "out");
    if (st == LIK_OK) st = check_scale(scale);
    if (st != LIK_OK) return st;
    int dev = 0;
    if ((st = check_device(&dev)) != LIK_OK) return st;
    const int64_t codes = pages * heads * page_size * dim, B = requests;
    const int64_t q_span = span(rows, q_token_stride, q_heads, q_head_stride, dim);
    const int64_t out_span = span(rows, out_token_stride, q_heads, out_head_stride, dim);
    const int64_t table = B > 0 && table_cols > 0 ? (B - 1) * table_stride + table_cols : 0;
    const Spec specs[] = {
        {"q", q, true, q_span},
        {"k_cache", k_cache, true, codes},
        {"v_cache", v_cache, true, codes},
        {"k_scale", k_scale, true, pages * heads},
        {"v_scale", v_scale, true, pages * heads},
        {"block_table", block_table, true, table},
        {"offsets", offsets, true, B + 1},
        {"lengths", lengths, true, B},
        {"out", out, true, out_span},
        {"lse", lse, false, rows * q_heads},
    };
    if ((st = check_buffers(dev, specs, 10)) != LIK_OK) return st;
    if ((st = check_aligned(q, 2, "q")) != LIK_OK || (st = check_aligned(out, 2, "out")) != LIK_OK) return st;
    if ((st = check_aligned(k_cache, 16, "k_cache")) != LIK_OK || (st = check_aligned(v_cache, 16, "v_cache")) != LIK_OK)
        return st;
    for (int i = 3; i < 10; ++i)
        if (i != 8 && (st = check_aligned(specs[i].ptr, 4, specs[i].name)) != LIK_OK) return st;
    if (rows == 0 || requests == 0) return LIK_OK;
    const size_t need = cache_attention_workspace(rows, q_heads, heads, dim, requests, max_added);
    if ((st = check_workspace(workspace, workspace_bytes, need, dev)) != LIK_OK) return st;
    const Bytes ins[] = {{"q", q, 2 * q_span},
                         {"k_cache", k_cache, codes},
                         {"v_cache", v_cache, codes},
                         {"k_scale", k_scale, 4 * pages * heads},
                         {"v_scale", v_scale, 4 * pages * heads},
                         {"block_table", block_table, 4 * table},
                         {"offsets", offsets, 4 * (B + 1)},
                         {"lengths", lengths, 4 * B}};
    const Bytes outs[] = {{"out", out, 2 * out_span},
                          {"lse", lse, 4 * rows * q_heads},
                          {"workspace", workspace, static_cast<int64_t>(need)}};
    if ((st = check_apart(outs, 3, ins, 8)) != LIK_OK) return st;
    a.q = q;
    a.dtype = static_cast<int>(dtype);
    a.rows = rows;
    a.q_heads = static_cast<int>(q_heads);
    a.heads = static_cast<int>(heads);
    a.dim = static_cast<int>(dim);
    a.q_token_stride = q_token_stride;
    a.q_head_stride = q_head_stride;
    a.k_cache = static_cast<const uint8_t*>(k_cache);
    a.v_cache = static_cast<const uint8_t*>(v_cache);
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    a.pages = pages;
    a.table = block_table;
    a.cols = table_cols;
    a.stride = table_stride;
    a.offsets = offsets;
    a.lengths = lengths;
    a.requests = static_cast<int>(requests);
    a.max_added = max_added;
    a.scale = scale;
    a.out = out;
    a.out_token_stride = out_token_stride;
    a.out_head_stride = out_head_stride;
    a.lse = lse;
    a.workspace = workspace;
    const cudaError_t e = launch_cache_attention(a, stream);
    return e == cudaSuccess ? LIK_OK : cuda_fail(e, "cache attention launch");
}

static lik_status check_verify(int64_t drafts, int64_t requests, int64_t cols) {
    lik_status st = check_requests(requests);
    if (st != LIK_OK) return st;
    if (drafts < 0 || cols < 0) return fail(LIK_ERR_INVALID_ARG, "negative size");
    if (cols < 1) return fail(LIK_ERR_INVALID_ARG, "cols must be >= 1");
    if (drafts > (int64_t(1) << 20)) return fail(LIK_ERR_UNSUPPORTED, "drafts %lld > 2^20", static_cast<ll>(drafts));
    if (cols > (int64_t(1) << 30)) return fail(LIK_ERR_UNSUPPORTED, "cols %lld > 2^30", static_cast<ll>(cols));
    return LIK_OK;
}

extern "C" lik_status lik_verify_drafts_workspace_bytes(int64_t drafts, int64_t requests, int64_t cols,
                                                        size_t* bytes) {
    clear_message();
    if (!bytes) return fail(LIK_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    const lik_status st = check_verify(drafts, requests, cols);
    if (st != LIK_OK || requests == 0) return st;
    *bytes = verify_workspace(drafts, requests, cols);
    return LIK_OK;
}

extern "C" lik_status lik_verify_drafts(const void* target_logits, const void* draft_logits, lik_dtype dtype,
                                        int64_t drafts, int64_t requests, int64_t cols, int64_t target_stride,
                                        int64_t draft_stride, const int32_t* drafted, const int32_t* offsets,
                                        const float* uniform, const float* noise, float scale, int32_t* tokens,
                                        int32_t* accepted, float* logp, void* workspace, size_t workspace_bytes,
                                        cudaStream_t stream) {
    clear_message();
    if (!known_dtype(dtype)) return fail(LIK_ERR_INVALID_ARG, "unknown dtype %d", static_cast<int>(dtype));
    lik_status st = check_verify(drafts, requests, cols);
    if (st == LIK_OK) st = check_scale(scale);
    if (st != LIK_OK) return st;
    const int64_t rows = drafts + requests, es = static_cast<int64_t>(elem_bytes(dtype));
    if (target_stride < cols || (draft_logits && draft_stride < cols))
        return fail(LIK_ERR_INVALID_ARG, "a row stride is below cols %lld", static_cast<ll>(cols));
    if (target_stride > (int64_t(1) << 31) || (draft_logits && draft_stride > (int64_t(1) << 31)))
        return fail(LIK_ERR_UNSUPPORTED, "a row stride is above 2^31");
    if (requests == 0 && drafts > 0) return fail(LIK_ERR_INVALID_ARG, "drafts without a request");
    int dev = 0;
    if ((st = check_device(&dev)) != LIK_OK) return st;
    const int64_t t_span = rows > 0 ? (rows - 1) * target_stride + cols : 0;
    const int64_t d_span = drafts > 0 ? (drafts - 1) * draft_stride + cols : 0;
    const Spec specs[] = {
        {"target_logits", target_logits, true, t_span},
        {"draft_logits", draft_logits, false, d_span},
        {"drafted", drafted, true, drafts},
        {"offsets", offsets, requests > 0, requests + 1},
        {"uniform", uniform, true, drafts},
        {"noise", noise, true, requests * cols},
        {"tokens", tokens, true, rows},
        {"accepted", accepted, true, requests},
        {"logp", logp, true, rows},
    };
    if ((st = check_buffers(dev, specs, 9)) != LIK_OK) return st;
    if ((st = check_aligned(target_logits, es, "target_logits")) != LIK_OK) return st;
    if ((st = check_aligned(draft_logits, es, "draft_logits")) != LIK_OK) return st;
    for (int i = 2; i < 9; ++i)
        if ((st = check_aligned(specs[i].ptr, 4, specs[i].name)) != LIK_OK) return st;
    if (requests == 0) return LIK_OK;
    const size_t need = verify_workspace(drafts, requests, cols);
    if ((st = check_workspace(workspace, workspace_bytes, need, dev)) != LIK_OK) return st;
    const Bytes ins[] = {{"target_logits", target_logits, t_span * es},
                         {"draft_logits", draft_logits, d_span * es},
                         {"drafted", drafted, 4 * drafts},
                         {"offsets", offsets, 4 * (requests + 1)},
                         {"uniform", uniform, 4 * drafts},
                         {"noise", noise, 4 * requests * cols}};
    const Bytes outs[] = {{"tokens", tokens, 4 * rows},
                          {"accepted", accepted, 4 * requests},
                          {"logp", logp, 4 * rows},
                          {"workspace", workspace, static_cast<int64_t>(need)}};
    if ((st = check_apart(outs, 4, ins, 6)) != LIK_OK) return st;
    VerifyArgs a{};
    a.target = target_logits;
    a.draft = draft_logits;
    a.dtype = static_cast<int>(dtype);
    a.drafts = drafts;
    a.requests = static_cast<int>(requests);
    a.cols = cols;
    a.target_stride = target_stride;
    a.draft_stride = draft_stride;
    a.drafted = drafted;
    a.offsets = offsets;
    a.uniform = uniform;
    a.noise = noise;
    a.scale = scale;
    a.tokens = tokens;
    a.accepted = accepted;
    a.logp = logp;
    a.workspace = workspace;
    const cudaError_t e = launch_verify(a, stream);
    return e == cudaSuccess ? LIK_OK : cuda_fail(e, "draft verification launch");
}
