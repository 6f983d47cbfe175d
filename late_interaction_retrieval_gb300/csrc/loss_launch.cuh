// loss_launch.cuh -- the instances of the row kernels for one type of logits.
#pragma once

#include "loss_rows.cuh"
#include "loss_short.cuh"

namespace lik {
namespace loss {

// Rows of up to 1 KB take a warp each.  Above, a block is faster (8192 rows of
// bf16, a step with the sum: 4 KB 18 us, 21 by a warp of 8 granules a lane;
// distillation 24 and 35).
template <typename T, int kHead, int kForm>
cudaError_t launch_form(const LossRows& L, bool* summed, cudaStream_t stream) {
    if (L.cols * static_cast<int64_t>(sizeof(T)) <= kShortBytes) return launch_short<T, kHead, kForm>(L, summed, stream);
    return launch_rows_kernel<T, kHead, kForm>(L, stream);
}

template <typename T>
cudaError_t launch_rows(LossHead head, LossForm form, const LossRows& L, bool* summed, cudaStream_t stream) {
    if (head == kHeadDistill) {
        if (form == kFwd) return launch_form<T, kHeadDistill, kFwd>(L, summed, stream);
        if (form == kBwd) return launch_form<T, kHeadDistill, kBwd>(L, summed, stream);
        return launch_form<T, kHeadDistill, kStep>(L, summed, stream);
    }
    // the gradient of a target head comes from its row states alone
    if (form == kBwd) return launch_form<T, kHeadToken, kBwd>(L, summed, stream);
    if (head == kHeadToken) return launch_form<T, kHeadToken, kFwd>(L, summed, stream);
    if (form == kFwd) return launch_form<T, kHeadPolicy, kFwd>(L, summed, stream);
    return launch_form<T, kHeadPolicy, kStep>(L, summed, stream);
}

}  // namespace loss
}  // namespace lik
