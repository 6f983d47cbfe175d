// loss_launch.cuh -- the instances of the row kernel for one type of logits.
#pragma once

#include "loss_rows.cuh"
#include "loss_short.cuh"

namespace lik {
namespace loss {

// Two CTAs of 8 consumer warps share an SM, or four of 4.  A CTA takes a row
// from its loads to its stores in some 3 us, mostly latency, so short rows want
// more CTAs (8192 rows of bf16, a step: 16 KB rows 73 us with four CTAs, 87 with
// two; 32 KB 117 and 121).  Two hold up to 64 KB of a row each, four up to 32 KB:
// longer rows take two (64 KB: 185 us, 274 with four).  The forms with one pass
// over the logits hold nothing: forward four are as good or better throughout
// (64 KB rows 91 us and 95), for the gradient two are better where rows are long
// (bf16 4096 x 32000, forward and gradient: 150 us, 161 with four).  Teachers of
// many entries leave four too little room.
template <typename T, int kHead, int kForm>
cudaError_t launch_form(const LossRows& L, bool* summed, unsigned int* err, cudaStream_t stream) {
    // up to 4 KB (and the loose elements): a warp a row, in registers
    constexpr int64_t kV = 16 / sizeof(T);
    if (L.cols <= 64 * kV) return launch_short<T, kHead, kForm, 2>(L, summed, stream);
    if (L.cols <= 256 * kV) return launch_short<T, kHead, kForm, 8>(L, summed, stream);
    const RingConfig four = ring_config<kHead, kForm, 4, 4, 4>(L, 1);
    const int64_t row_bytes = L.cols * static_cast<int64_t>(sizeof(T));
    const int64_t most = kForm == kFwd ? INT64_MAX : kForm == kStep ? four.hold * int64_t(8192) : 32768;
    if (four.slots >= 4 && row_bytes <= most) return launch_ring<T, kHead, kForm, 4, 4, 4>(L, err, stream);
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
