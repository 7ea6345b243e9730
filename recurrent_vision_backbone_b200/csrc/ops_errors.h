// ops_errors.h -- how the operators around the token mixer report errors through gtr_gla.cu.
#pragma once

#include <cuda_runtime.h>

#include "../../include/gtr_ops.h"

namespace gtr {

// Defined in gtr_gla.cu: keeps the error for gtr_gla_last_error and turns it into a status.
gtr_status_t ops_cuda_status(cudaError_t e);
// Error bits of one source file's kernels on the current device, read and cleared
// (gtr_gla_device_status collects them). kOpsErrCuda: the word could not be read.
constexpr unsigned kOpsErrRange = 2u, kOpsErrCuda = 0x80000000u;
unsigned conv_take_errors();
unsigned ssm_take_errors();
unsigned ssm_bwd_take_errors();
unsigned norm_take_errors();

}  // namespace gtr
