// row_io.cuh -- 16 consecutive row elements per thread: loads and stores shared by the
// layer operators' kernels (BF16 or FP32 rows, widened to FP32).
//
// A row may start at any element.  `grain` is the widest access that every full
// 16-element chunk of the tensor allows (32 or 16 bytes, 0 for element accesses), the
// same for the whole tensor, so the choice is one uniform branch: 32-byte accesses move
// whole sectors (one request of a warp covers 1 KB), and an odd row length falls back
// to elements.  A chunk cut by the row's end is always moved element by element.
#pragma once

#include <cuda_bf16.h>

#include "device_common.cuh"

namespace nvfp4 {

constexpr int kChunk = 16;  // elements per thread and access group

// Launch a kernel whose set-up may overlap the end of the one before it in the stream; it
// begins with pdl_wait().
template <typename... P>
inline cudaError_t launch_after(void (*kernel)(P...), unsigned grid, unsigned threads,
                                cudaStream_t stream, const P&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The grain of rows of `cols` elements of `elem` bytes at p.
inline int row_grain(const void* p, int64_t cols, int elem) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p) | (uintptr_t)(cols * elem);
  return a % 32 == 0 ? 32 : (a % 16 == 0 ? 16 : 0);
}

__device__ __forceinline__ void ldg_v8(const void* p, uint32_t* w) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                 "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}
__device__ __forceinline__ void ldg_v4(const void* p, uint32_t* w) {
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "l"(p));
}

__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// One chunk as it lies in memory: 8 words of BF16 pairs or 16 FP32 words; elements from n
// on are zero.
template <bool BF16>
struct Chunk {
  static constexpr int kWords = BF16 ? 8 : 16;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const void* base, int64_t off, int n, int grain) {
    const char* p = static_cast<const char*>(base) + off * (BF16 ? 2 : 4);
    if (n == kChunk && grain == 32) {
#pragma unroll
      for (int i = 0; i < kWords; i += 8) ldg_v8(p + 4 * i, w + i);
    } else if (n == kChunk && grain == 16) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) ldg_v4(p + 4 * i, w + i);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = 0;
      if constexpr (BF16) {
        const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
        for (int i = 0; i < kChunk; ++i)
          if (i < n) w[i >> 1] |= (uint32_t)q[i] << (16 * (i & 1));
      } else {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(p);
#pragma unroll
        for (int i = 0; i < kChunk; ++i)
          if (i < n) w[i] = q[i];
      }
    }
  }
  // From a row held in shared memory, 16-byte aligned (so n is a whole number of 16-byte
  // units).  Lanes are 32 or 64 bytes apart; rotating the order of a lane's units spreads
  // the eight lanes of an access over all banks.
  __device__ __forceinline__ void load_shared(const uint8_t* p, int n, int lane) {
    constexpr int kUnits = kWords / 4;
    const int rot = BF16 ? (lane >> 2) & 1 : (lane >> 1) & 3;
    uint4 u[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const int at = (k + rot) & (kUnits - 1);
      u[k] = at * (kChunk / kUnits) < n ? *reinterpret_cast<const uint4*>(p + 16 * at)
                                        : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int d = 1; d < kUnits; d *= 2) {  // u[k] holds unit k + rot: rotate back
      uint4 r[kUnits];
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        const uint4 a = u[k], b = u[(k - d) & (kUnits - 1)];
        r[k].x = (rot & d) ? b.x : a.x;
        r[k].y = (rot & d) ? b.y : a.y;
        r[k].z = (rot & d) ? b.z : a.z;
        r[k].w = (rot & d) ? b.w : a.w;
      }
#pragma unroll
      for (int k = 0; k < kUnits; ++k) u[k] = r[k];
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      w[4 * k] = u[k].x;
      w[4 * k + 1] = u[k].y;
      w[4 * k + 2] = u[k].z;
      w[4 * k + 3] = u[k].w;
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (BF16) return (i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
    else return __uint_as_float(w[i]);
  }
  // Round 16 values into the chunk (nearest even).
  __device__ __forceinline__ void set(const float* v) {
    if constexpr (BF16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = bf16x2_bits(v[2 * i], v[2 * i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(v[i]);
    }
  }
  __device__ __forceinline__ void store(void* base, int64_t off, int n, int grain) const {
    char* p = static_cast<char*>(base) + off * (BF16 ? 2 : 4);
    if (n == kChunk && grain == 32) {
#pragma unroll
      for (int i = 0; i < kWords; i += 8) stg_v8(p + 4 * i, w + i);
    } else if (n == kChunk && grain == 16) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4)
        *reinterpret_cast<uint4*>(p + 4 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    } else if constexpr (BF16) {
      uint16_t* q = reinterpret_cast<uint16_t*>(p);
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        if (i < n) q[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    } else {
      uint32_t* q = reinterpret_cast<uint32_t*>(p);
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        if (i < n) q[i] = w[i];
    }
  }
};

// The 16 FP32 values of a chunk of a BF16 or FP32 vector (type known at run time).
__device__ __forceinline__ void load_vector16(const void* base, bool bf16, int64_t off, int n,
                                              int grain, float* v) {
  if (bf16) {
    Chunk<true> c;
    c.load(base, off, n, grain);
#pragma unroll
    for (int i = 0; i < kChunk; ++i) v[i] = c.get(i);
  } else {
    Chunk<false> c;
    c.load(base, off, n, grain);
#pragma unroll
    for (int i = 0; i < kChunk; ++i) v[i] = c.get(i);
  }
}

// Contiguous bytes to shared memory, completing on `bar` (16-byte aligned addresses, size a
// multiple of 16).
__device__ __forceinline__ void bulk_copy_in(void* dst, const void* src, uint32_t bytes,
                                             uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_addr(bar))
      : "memory");
}

// Elements of the chunk that starts at column c of a row of `cols` (0 past its end).
__device__ __forceinline__ int chunk_len(int64_t c, int64_t cols) {
  const int64_t left = cols - c;
  return left >= kChunk ? kChunk : (left > 0 ? (int)left : 0);
}

}  // namespace nvfp4
