// What the translation units of the library share on the host side (defined in dg_api.cu).
#pragma once
#include <cuda_runtime.h>

namespace dg {

// Sets the message of dg_last_error and returns `code`.
int fail(int code, const char *fmt, ...);
int cuda_fail(cudaError_t e, const char *what);
// Checks that the current device is an sm_100 and gives its index and SM count under the cap of dg_set_num_sms.
int current_device(int &device, int &num_sms);
// The library's stream-ordered memory pool of a device.
int scratch_pool(int device, cudaMemPool_t &pool);
// The error word of the current device (nullptr if it cannot be had).
unsigned *device_error_word();
// Segment alignment of the contiguous layout now in force (128 or 256).
int contiguous_alignment();

}  // namespace dg
