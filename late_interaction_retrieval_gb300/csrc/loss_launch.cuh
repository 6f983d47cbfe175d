// loss_launch.cuh -- the instances of the row kernel for one type of logits.
#pragma once

#include "loss_block.cuh"
#include "loss_rows.cuh"
#include "loss_short.cuh"

namespace lik {
namespace loss {

// By the length of a row (bf16 unless said, 8192 rows of logits, a step with the
// sum, inputs beyond L2):
//   to 1 KB   a warp a row, its granules in registers;
//   to 40 KB  a block a row, likewise: 4 KB rows 18 us (21 by a warp a row of 8
//             granules a lane; distillation 24 and 35), 8 KB 28 (53 through the
//             ring), 16 KB 48 (74), 32 KB 90 (109), 40 KB 117 (149); forward 8 KB
//             18 (33), 16 KB 28 (41), 32 KB 51 (57), 40 KB 65 (64).  Few blocks of
//             longer rows fit an SM's registers, and their latencies show: 48 KB
//             153 (151), 64 KB 234 (181);
//   longer    through the ring, by CTAs that share an SM: two of 8 consumer warps,
//             which hold up to 64 KB of a row each between a step's passes.  A
//             forward holds nothing, and four CTAs of 4 warps are as good or better
//             throughout (64 KB rows 91 us and 95); teachers of many entries leave
//             four too little room.
template <typename T, int kHead, int kForm>
cudaError_t launch_form(const LossRows& L, bool* summed, unsigned int* err, cudaStream_t stream) {
    const int64_t row_bytes = L.cols * static_cast<int64_t>(sizeof(T));
    if (row_bytes <= kShortBytes) return launch_short<T, kHead, kForm>(L, summed, stream);
    if (row_bytes <= kBlockBytes) return launch_block<T, kHead, kForm>(L, stream);
    if constexpr (kForm == kFwd) {
        if (ring_config<kHead, kForm, 4, 4, 4>(L, 1).slots >= 4) return launch_ring<T, kHead, kForm, 4, 4, 4>(L, err, stream);
    }
    return launch_ring<T, kHead, kForm, 8, 4, 2>(L, err, stream);
}

template <typename T>
cudaError_t launch_rows(LossHead head, LossForm form, const LossRows& L, bool* summed, cudaStream_t stream) {
    unsigned int* err = device_error_word();
    if (!err) return cudaErrorInvalidDevice;
    if (head == kHeadDistill) {
        if (form == kFwd) return launch_form<T, kHeadDistill, kFwd>(L, summed, err, stream);
        if (form == kBwd) return launch_form<T, kHeadDistill, kBwd>(L, summed, err, stream);
        return launch_form<T, kHeadDistill, kStep>(L, summed, err, stream);
    }
    // the gradient of a target head comes from its row states alone
    if (form == kBwd) return launch_form<T, kHeadToken, kBwd>(L, summed, err, stream);
    if (head == kHeadToken) return launch_form<T, kHeadToken, kFwd>(L, summed, err, stream);
    if (form == kFwd) return launch_form<T, kHeadPolicy, kFwd>(L, summed, err, stream);
    return launch_form<T, kHeadPolicy, kStep>(L, summed, err, stream);
}

}  // namespace loss
}  // namespace lik
