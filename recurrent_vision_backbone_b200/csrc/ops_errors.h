// ops_errors.h -- how the operators around the token mixer report errors through gtr_gla.cu.
#pragma once

#include <cuda_runtime.h>

#include "../../include/gtr_ops.h"

namespace gtr {

// Defined in gtr_gla.cu: keeps the error for gtr_gla_last_error and turns it into a status.
gtr_status_t ops_cuda_status(cudaError_t e);
// The error words of the source files' kernels: their addresses on the current device, null where it cannot
// be had (gtr_gla_device_status collects and clears them).
constexpr unsigned kOpsErrRange = 2u;
unsigned *conv_error_word();
unsigned *ssm_error_word();
unsigned *ssm_bwd_error_word();
unsigned *norm_error_word();

}  // namespace gtr
