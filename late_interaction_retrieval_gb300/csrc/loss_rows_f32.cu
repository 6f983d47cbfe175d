// loss_rows_f32.cu -- the row kernel of the training objectives, f32 logits.
#include "loss_launch.cuh"

namespace lik {
cudaError_t launch_loss_f32(LossHead head, LossForm form, const LossRows& L, bool* summed, cudaStream_t stream) {
    return loss::launch_rows<float>(head, form, L, summed, stream);
}
}  // namespace lik
