// row_ring.cuh -- what the norm's forward and backward kernels share: the reduction over a
// row's team of threads, and the shared-memory ring that rows run through.
#pragma once

#include <algorithm>

#include "internal.h"
#include "row_io.cuh"

namespace nvfp4 {
namespace {

// Sum and maximum over the TPR threads of a row's team; every thread gets both.  The
// order of the sum depends on TPR alone.  red: one pair per warp, in two buffers used in
// turn, so that one barrier per row is enough.  BARRIER: with the CTA's barrier also where
// a team is one warp.
template <int TPR, bool BARRIER = false>
__device__ __forceinline__ float2 team_sum_max(float s, float m, float2* red) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, d));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  }
  if constexpr (TPR > 32) {
    constexpr int kWarps = TPR / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) red[warp] = make_float2(s, m);
    __syncthreads();
    constexpr int kTree = kWarps <= 2 ? 2 : kWarps <= 4 ? 4 : kWarps <= 8 ? 8 : kWarps <= 16 ? 16 : 32;
    const int i = lane % kTree;
    const float2 v = i < kWarps ? red[warp - warp % kWarps + i] : make_float2(0.0f, 0.0f);
    s = v.x;
    m = v.y;
#pragma unroll
    for (int d = kTree / 2; d > 0; d >>= 1) {
      s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, d));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    }
  } else if constexpr (BARRIER) {
    __syncthreads();
  }
  return make_float2(s, m);
}

// ---------------------------------------------------------------- a ring of rows

// Many aligned rows: they run through a ring in shared memory, filled by bulk copies that
// thread 0 issues several rows ahead, so that the row's barrier and its arithmetic never
// leave the memory idle, whatever the registers allow to be resident.  A stage holds one
// group of kTeams consecutive rows of each tensor (consecutive in memory: one copy each).
// The row's reduction barrier is also what frees its stage: by then every thread has the
// stage's values in registers.
constexpr int kRingStages = 8;

struct RingArgs {
  int stages;
  int tensor_bytes;  // stride of a stage's tensors
  int stage_bytes;
};

// ANY: rows of any length and alignment within their tensors, whose bases are 16-byte aligned:
// a stage receives the 16-byte units that cover the group, and the group starts `shift`
// bytes into it.  The units never reach past the tensor: its last few bytes, if they fill
// no unit, are copied by the threads (finish()).  They belong to the last group alone: a
// group of several teams starts on a unit, or its rows are longer than one.
template <int NT, bool ANY = false>
struct RowRing {
  uint64_t* full;
  int* err;
  uint8_t* smem;
  const void* src[NT];
  int64_t rows, row_bytes;
  int teams;
  RingArgs g;

  __device__ __forceinline__ uint8_t* stage(int s) const { return smem + s * g.stage_bytes; }
  // thread 0: start the copies of the group of rows that begins at row0
  __device__ __forceinline__ void fetch(int s, int64_t row0) const {
    const int64_t left = rows - row0;
    int64_t from = row0 * row_bytes, to = from + (left < teams ? left : teams) * row_bytes;
    if constexpr (ANY) {
      from &= ~(int64_t)15;
      const int64_t end = (rows * row_bytes) & ~(int64_t)15;
      to = (to + 15) & ~(int64_t)15;
      if (to > end) to = end > from ? end : from;
    }
    const uint32_t bytes = (uint32_t)(to - from);
    int n = 0;
#pragma unroll
    for (int i = 0; i < NT; ++i) n += src[i] != nullptr;
    mbar_expect_tx(&full[s], bytes * n);
#pragma unroll
    for (int i = 0; i < NT; ++i)
      if (src[i] != nullptr)
        if (!ANY || bytes > 0)
          bulk_copy_in(stage(s) + i * g.tensor_bytes, static_cast<const char*>(src[i]) + from,
                       bytes, &full[s]);
  }
  // ANY: where in its stage the group of rows at row0 starts.
  __device__ __forceinline__ int shift(int64_t row0) const {
    return ANY ? (int)((row0 * row_bytes) & 15) : 0;
  }
  // ANY, every thread, after wait(): the tensor's last bytes, which no unit holds, into the
  // stage of the group that ends with them.
  __device__ __forceinline__ void finish(int s, int64_t row0) const {
    if constexpr (ANY) {
      const int64_t total = rows * row_bytes, end = total & ~(int64_t)15;
      if (row0 + teams < rows || end == total) return;  // the same for the whole CTA
      const int64_t from = (row0 * row_bytes) & ~(int64_t)15;
      const int n = (int)(total - end);
#pragma unroll
      for (int i = 0; i < NT; ++i)
        if (src[i] != nullptr && (int)threadIdx.x < n)
          stage(s)[i * g.tensor_bytes + (end - from) + threadIdx.x] =
              static_cast<const uint8_t*>(src[i])[end + threadIdx.x];
      __syncthreads();
    }
  }
  __device__ __forceinline__ void start(int64_t step) const {
    if (threadIdx.x == 0) {
      for (int s = 0; s < g.stages; ++s) mbar_init(&full[s], 1);
      *err = 0;
      fence_mbar_init();
      for (int s = 0; s < g.stages; ++s) {
        const int64_t row0 = (int64_t)blockIdx.x * teams + s * step;
        if (row0 < rows) fetch(s, row0);
      }
    }
    __syncthreads();
  }
  // Wait for use `it` of the ring; false (with the error noted) if it gave up.
  __device__ __forceinline__ bool wait(int s, int it) const {
    const bool ok = mbar_wait_bounded(&full[s], (it / g.stages) & 1);
    if (!ok) *err = 1;
    return ok;
  }
  // After a timeout: thread 0 waits (bounded) for the copies still in flight.
  __device__ __forceinline__ void give_up(int it, int64_t row0, int64_t step, int* status) const {
    if (threadIdx.x != 0) return;
    raise_status(status, kStatusTimeout);
    for (int k = 0; k < g.stages; ++k)
      if (row0 + k * step < rows)
        mbar_wait_bounded(&full[(it + k) % g.stages], ((it + k) / g.stages) & 1);
  }
};

template <typename K>
int resident_ctas(K kernel, int threads) {
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0) != cudaSuccess) {
    cudaGetLastError();
    n = 1;
  }
  return std::max(1, n);
}

// A ring kernel's CTAs per SM by registers, and its static shared memory.
constexpr int kCtaSmem = 227 << 10;  // shared memory that one CTA may have
struct RingKernel {
  int resident;
  int static_bytes;
};
template <typename K>
RingKernel ring_kernel(K kernel, int threads) {
  cudaFuncAttributes f;
  if (cudaFuncGetAttributes(&f, kernel) != cudaSuccess) {
    cudaGetLastError();
    return {0, 0};
  }
  return {resident_ctas(kernel, threads), (int)f.sharedSizeBytes};
}
template <typename K>
cudaError_t allow_ring(K kernel, const RingKernel& k) {  // on the current device
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kCtaSmem - k.static_bytes);
}

// CTAs per SM and the ring of each: as many CTAs as the registers allow while each keeps
// at least two stages.  ctas == 0: two stages do not fit, or there is nothing to hold (rows
// without columns).
struct RingPlan {
  int ctas;
  RingArgs g;
};
RingPlan plan_ring(const RingKernel& k, int tensors, int64_t group_bytes, bool any = false) {
  RingPlan p{};
  if (group_bytes <= 0) return p;
  // any: up to 30 bytes of the units around the rows, and a lane's reads past a row's end
  const int64_t tensor = (group_bytes + (any ? 128 : 0) + 127) / 128 * 128, stage = tensors * tensor;
  for (int c = k.resident; c > 0; --c) {
    // an SM's 228 KB, of which every CTA takes 1 KB beside its own
    const int64_t room =
        std::min<int64_t>(kCtaSmem, (228 << 10) / c - (1 << 10)) - k.static_bytes;
    if (room < 2 * stage) continue;
    p.ctas = c;
    p.g.stages = (int)std::min<int64_t>(kRingStages, room / stage);
    p.g.tensor_bytes = (int)tensor;
    p.g.stage_bytes = (int)stage;
    break;
  }
  return p;
}

}  // namespace
}  // namespace nvfp4
