// loss_rows_bf16.cu -- the row kernel of the training objectives, bf16 logits.
#include "loss_launch.cuh"

namespace lik {
cudaError_t launch_loss_bf16(LossHead head, LossForm form, const LossRows& L, bool* summed, cudaStream_t stream) {
    return loss::launch_rows<__nv_bfloat16>(head, form, L, summed, stream);
}
}  // namespace lik
