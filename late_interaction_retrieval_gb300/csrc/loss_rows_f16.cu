// loss_rows_f16.cu -- the row kernel of the training objectives, f16 logits.
#include "loss_launch.cuh"

namespace lik {
cudaError_t launch_loss_f16(LossHead head, LossForm form, const LossRows& L, bool* summed, cudaStream_t stream) {
    return loss::launch_rows<__half>(head, form, L, summed, stream);
}
}  // namespace lik
