// api_common.h -- what the C ABI's translation units share: status reporting, argument
// checks and the current device.  Host side only, not part of the ABI.
#pragma once

#include <initializer_list>
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

// rows x 2 cols: the two halves of a gated product
inline nvfp4_status check_gated_sizes(int64_t rows, int64_t cols) {
  const nvfp4_status st = check_sizes(rows, cols);
  if (st != NVFP4_OK) return st;
  if (cols >= (1LL << 30)) return fail(NVFP4_ERR_INVALID, "twice the columns must be < 2^31");
  return NVFP4_OK;
}

inline bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

inline int64_t elem_bytes(int32_t dtype) { return dtype == NVFP4_IN_BF16 ? 2 : 4; }

// Every pointer that is given must be aligned to its element.
inline nvfp4_status check_elems(std::initializer_list<const void*> ptrs, int32_t dtype) {
  for (const void* p : ptrs)
    if (!aligned(p, elem_bytes(dtype)))
      return fail(NVFP4_ERR_INVALID, "a tensor is not aligned to its element size");
  return NVFP4_OK;
}

inline nvfp4_status check_workspace(const void* workspace, uint64_t have, uint64_t need) {
  if (need == 0) return NVFP4_OK;
  if (workspace == nullptr || !aligned(workspace, 16))
    return fail(NVFP4_ERR_INVALID, "workspace must be non-NULL and 16-byte aligned");
  if (have < need)
    return fail(NVFP4_ERR_INVALID,
                "workspace of " + std::to_string(have) + " bytes, " + std::to_string(need) +
                    " needed");
  return NVFP4_OK;
}

// Whether out shares bytes with in without starting where it starts (an element written
// before another thread reads it).
inline bool shifted(const void* out, const void* in, uint64_t bytes) {
  return out != in && bytes_overlap(out, bytes, in, bytes);
}

}  // namespace nvfp4
