// cache_attention.cu -- attention of a batch's new tokens over the 8-bit
// cache: which kernel takes a call.
#include "cache_attention.h"

namespace lik {

size_t cache_attention_workspace(int64_t, int64_t, int64_t, int64_t dim, int64_t, int64_t) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    return attention_split_workspace(dim, device_info(dev).sm_count);
}

cudaError_t launch_cache_attention(const AttentionArgs& a, cudaStream_t stream) {
    return launch_attention_split(a, stream);
}

}  // namespace lik
