// sector.cuh -- what the activations' backward kernels share: 32 bytes of a row per lane, the
// maxima of stored words, and the join of partial column sums and maxima.
#pragma once

#include "internal.h"
#include "row_io.cuh"

namespace nvfp4 {
namespace {

// 32 bytes of a row (W words, 8 or 4), one lane's columns: 16 BF16 or 8 FP32.
template <bool BF16, int W = 8>
struct Sector {
  static constexpr int kCols = BF16 ? 2 * W : W;
  uint32_t w[W];
  __device__ __forceinline__ void load(const void* base, int64_t off, int n, int grain) {
    const char* p = static_cast<const char*>(base) + off * (BF16 ? 2 : 4);
    if (W == 8 && n == kCols && grain == 32) {
      ldg_v8(p, w);
    } else if (n == kCols && grain >= 16) {
#pragma unroll
      for (int i = 0; i < W; i += 4) ldg_v4(p + 4 * i, w + i);
    } else {
#pragma unroll
      for (int i = 0; i < W; ++i) w[i] = 0;
#pragma unroll
      for (int i = 0; i < kCols; ++i)
        if (i < n) {
          if constexpr (BF16)
            w[i >> 1] |= (uint32_t) reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
          else
            w[i] = reinterpret_cast<const uint32_t*>(p)[i];
        }
    }
  }
  __device__ __forceinline__ void store(void* base, int64_t off, int n, int grain) const {
    char* p = static_cast<char*>(base) + off * (BF16 ? 2 : 4);
    if (W == 8 && n == kCols && grain == 32) {
      stg_v8(p, w);
    } else if (n == kCols && grain >= 16) {
#pragma unroll
      for (int i = 0; i < W; i += 4)
        *reinterpret_cast<uint4*>(p + 4 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < kCols; ++i)
        if (i < n) {
          if constexpr (BF16)
            reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
          else
            reinterpret_cast<uint32_t*>(p)[i] = w[i];
        }
    }
  }
  // The store of a warp whose lanes hold consecutive sectors (`run` columns exist from lane
  // 0's on), in rows whose grain does not allow 16-byte accesses.
  template <bool STAGED>
  __device__ __forceinline__ void store_warp(void* base, int64_t off, int n, int64_t run,
                                             int grain, uint8_t* smem, int lane) const {
    constexpr int kElem = BF16 ? 2 : 4;
    if (!STAGED || grain >= 16 || smem == nullptr) {
      store(base, off, n, grain);
      return;
    }
    staged_store<W, 4 * W, kElem, 8>(static_cast<char*>(base) + (off - (int64_t)kCols * lane) * kElem,
                        (int)run * kElem, grain, smem, lane, w);
  }
  // columns 2k and 2k + 1
  __device__ __forceinline__ Pair get(int k) const {
    if constexpr (BF16) return {bf16_lo(w[k]), bf16_hi(w[k])};
    else return {__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1])};
  }
  __device__ __forceinline__ void set(int k, Pair v) {
    if constexpr (BF16) {
      w[k] = bf16x2_bits(v.x, v.y);
    } else {
      w[2 * k] = __float_as_uint(v.x);
      w[2 * k + 1] = __float_as_uint(v.y);
    }
  }
};

// The load of such a warp: issue() for every tensor, settle() when the values are needed.
template <bool BF16, bool STAGED, int W = 8>
struct SectorLoad {
  Sector<BF16, W> s;
  StagedLoad<W, 4 * W, BF16 ? 2 : 4> raw;
  __device__ __forceinline__ void issue(const void* base, int64_t off, int n, int64_t run,
                                        int grain, const uint8_t* smem, int lane) {
    constexpr int kElem = BF16 ? 2 : 4;
    if (!STAGED || grain >= 16 || smem == nullptr) s.load(base, off, n, grain);
    else
      raw.issue(static_cast<const char*>(base) + (off - (int64_t)s.kCols * lane) * kElem, (int)run * kElem, grain, lane);
  }
  __device__ __forceinline__ const Sector<BF16, W>& settle(int grain, uint8_t* smem, int lane) {
    if constexpr (STAGED) {
      if (grain < 16 && smem != nullptr) raw.settle(grain, smem, lane, s.w);
    }
    return s;
  }
};

// max |a|, |b| of the values in a word (one FP32 or a pair of BF16), NaN skipped; the sign
// bits of the result mean nothing.
template <bool BF16>
__device__ __forceinline__ uint32_t word_absmax(uint32_t a, uint32_t b) {
  if constexpr (BF16) return absmax_bf16x2(a, b);
  return __float_as_uint(fmaxf(fabsf(__uint_as_float(a)), fabsf(__uint_as_float(b))));
}
template <bool BF16>
__device__ __forceinline__ float word_value(uint32_t a) {
  if constexpr (BF16) return bf16x2_hmax_f32(a);
  return __uint_as_float(a);
}

struct ActReduceArgs {
  const float* col_sum;
  const float* col_max;
  const float* row_max;
  float* dbias;
  float* col_amax;
  float* row_amax;
  int64_t rows, cols;
  int strips, row_parts;
  int col_ctas;
};

// The first col_ctas CTAs join 32 columns each (warp w the parts w, w + 8, ..., then the
// warps in turn), the others 256 rows each.
__global__ void __launch_bounds__(256) k_act_join(const ActReduceArgs a) {
  pdl_wait();
  if ((int)blockIdx.x < a.col_ctas) {
    __shared__ float s_sum[8][32], s_max[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float sum = 0.0f, mx = 0.0f;
    if (c < a.cols) {
#pragma unroll 4
      for (int p = warp; p < a.row_parts; p += 8) {
        if (a.dbias != nullptr) sum = __fadd_rn(sum, a.col_sum[(int64_t)p * a.cols + c]);
        if (a.col_amax != nullptr) mx = fmaxf(mx, a.col_max[(int64_t)p * a.cols + c]);
      }
    }
    s_sum[warp][lane] = sum;
    s_max[warp][lane] = mx;
    __syncthreads();
    if (warp == 0 && c < a.cols) {
#pragma unroll
      for (int i = 1; i < 8; ++i) {
        sum = __fadd_rn(sum, s_sum[i][lane]);
        mx = fmaxf(mx, s_max[i][lane]);
      }
      if (a.dbias != nullptr) a.dbias[c] = sum;
      if (a.col_amax != nullptr) a.col_amax[c] = mx;
    }
  } else {
    const int64_t r = (int64_t)(blockIdx.x - a.col_ctas) * 256 + threadIdx.x;
    if (r >= a.rows) return;
    float mx = 0.0f;
#pragma unroll 8
    for (int s = 0; s < a.strips; ++s) mx = fmaxf(mx, a.row_max[(int64_t)s * a.rows + r]);
    a.row_amax[r] = mx;
  }
}

// strips of 32 lanes: 512 BF16 or 256 FP32 columns (half of them with half sectors)
int64_t strips_of(int64_t cols, bool bf16, bool half = false) {
  const int strip = (bf16 ? 32 * Sector<true>::kCols : 32 * Sector<false>::kCols) / (half ? 2 : 1);
  return (cols + strip - 1) / strip;
}
int64_t round16(int64_t v) { return (v + 15) / 16 * 16; }

}  // namespace
}  // namespace nvfp4
