// The library's last-error message, shared by its translation units.
#pragma once

#include <cuda_runtime.h>

namespace moe {

// Record `msg` as the calling thread's last error and return `code`.
int set_error(int code, const char* msg);
// Record a failed CUDA call and return MOE_E_CUDA.
int set_cuda_error(cudaError_t e, const char* what);
// Forget the last error.
void clear_error();

}  // namespace moe
