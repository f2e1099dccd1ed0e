// api_common.h -- what the C ABI's translation units share: status reporting, argument
// checks and the current device.  Host side only, not part of the ABI.
#pragma once

#include <string>

#include "../../include/nvfp4.h"
#include "internal.h"

namespace nvfp4 {

// Record the message of a status for nvfp4_last_error and return the status.
nvfp4_status fail(nvfp4_status st, const std::string& msg);
nvfp4_status cuda_fail(cudaError_t e, const char* what);

// Whether the byte ranges [a, a + na) and [b, b + nb) share a byte.
bool bytes_overlap(const void* a, uint64_t na, const void* b, uint64_t nb);

nvfp4_status current_device(DeviceInfo* out);

bool valid_in_dtype(int32_t d);
nvfp4_status check_sizes(int64_t rows, int64_t cols);
nvfp4_status check_config(const nvfp4_config* cfg);
nvfp4_status check_out(const nvfp4_out* o, const char* name, int64_t lines, int64_t n,
                       int64_t amax_len);

inline bool valid_activation(int32_t act) {
  return act >= NVFP4_ACT_NONE && act <= NVFP4_ACT_SILU;
}

}  // namespace nvfp4
