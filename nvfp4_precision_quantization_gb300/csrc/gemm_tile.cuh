// gemm_tile.cuh -- how the tiled products' epilogues move blocks of 32 rows (one per lane) x 32
// columns.
#pragma once

#include "row_io.cuh"

namespace nvfp4 {

// 32 consecutive output columns of one row, FP32 -> D's type, in 32-byte (v8) or 16-byte
// stores.
__device__ __forceinline__ void store_run32(void* base, bool bf16, int64_t off, const float* v,
                                            bool v8) {
  const int step = bf16 ? 16 : 8;  // values of a 32-byte sector
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    uint32_t w[8];
    if (bf16) {
      if (g >= 2) break;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        w[j] = bf16x2_bits(v[(16 * g + 2 * j) & 31], v[(16 * g + 2 * j + 1) & 31]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[8 * g + j]);
    }
    char* dst = static_cast<char*>(base) + (off + g * step) * (bf16 ? 2 : 4);
    if (v8) {
      stg_v8(dst, w);
    } else {
      *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4*>(dst + 16) = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

// v[i] of lane l <- v[l] of lane i: a 32 x 32 transposition between the lanes of a warp.
__device__ __forceinline__ void transpose32(float* v, int lane) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const bool upper = lane & d;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if (i & d) continue;
      const float got = __shfl_xor_sync(0xffffffffu, upper ? v[i] : v[i | d], d);
      if (upper) v[i] = got;
      else v[i | d] = got;
    }
  }
}

}  // namespace nvfp4
