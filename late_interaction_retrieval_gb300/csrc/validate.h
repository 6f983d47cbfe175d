// validate.h -- argument checks shared by the C entry points (defined in api.cu).
#pragma once

#include <cstdint>

#include "lik.h"

namespace lik {

// Records a message for lik_last_error_message() and returns `s`.
lik_status fail(lik_status s, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
lik_status cuda_fail(cudaError_t e, const char* what);
void clear_message();

bool known_dtype(lik_dtype t);

// The current device must be a GB300 (sm_103).
lik_status check_device(int* dev_out);

// A non-NULL pointer must be device (or managed) memory of device `dev`.
lik_status check_pointer(const void* p, int dev, const char* name);

lik_status check_aligned(const void* p, uintptr_t bytes, const char* name);

struct Spec {
    const char* name;
    const void* ptr;
    bool required;  // must be non-NULL when the buffer has elements
    int64_t elems;
};
lik_status check_buffers(int dev, const Spec* specs, int n);

}  // namespace lik
