// cache_attention.cu -- attention of a batch's new tokens over the 8-bit
// cache: which kernel takes a call.
#include "cache_attention.h"

namespace lik {
namespace {

// Few rows a key head take the kernel whose tiles have 8 or 16 rows: it reads the cache once for each 16 rows, the other
// once for 256.  Measured, 64 requests of 4700 tokens, 8 key heads of 128, bf16 (fp16): 16 rows 183 us (203) here, 256
// (287) there; 20 rows 315 (352) and 257 (288).  4 requests of 75000 tokens: 16 rows 162 (180) and 239 (264), 20 rows
// 281 (302) and 241 (263).
bool few_rows(int64_t max_added, int64_t group) { return max_added * group <= 16; }

}  // namespace

size_t cache_attention_workspace(int64_t rows, int64_t q_heads, int64_t heads, int64_t dim, int64_t,
                                 int64_t max_added) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    const int sms = device_info(dev).sm_count;
    return few_rows(max_added, q_heads / heads) ? attention_split_workspace(dim, sms)
                                                : attention_wide_workspace(rows, q_heads / heads, dim, sms);
}

cudaError_t launch_cache_attention(const AttentionArgs& a, cudaStream_t stream) {
    return few_rows(a.max_added, a.q_heads / a.heads) ? launch_attention_split(a, stream)
                                                      : launch_attention_wide(a, stream);
}

}  // namespace lik
