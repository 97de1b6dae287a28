// The thread's last error (disco_last_error), for entry points outside capi.cu (internal).
#pragma once

#include <cuda_runtime.h>

#include "../../include/disco.h"

namespace disco {

disco_status set_error(disco_status s, const char* msg);
disco_status set_cuda_error(cudaError_t e, const char* where);

}  // namespace disco
