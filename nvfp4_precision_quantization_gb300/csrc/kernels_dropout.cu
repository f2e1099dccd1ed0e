// kernels_dropout.cu -- dropout with a mask that is made where it is used, and the residual's
// addition: y = residual + (kept ? x / (1 - p) : 0).  The gradient is the same call on dy.
//
// Bound by memory: two reads and a write (one read without a residual); a thread makes the 16
// elements of a chunk from two Philox blocks.  Measured: 16384 x 8192 BF16 with a residual 118 us, 6.8
// TB/s, the rate of a copy.
#include <algorithm>

#include "dropout.cuh"

namespace nvfp4 {
namespace {

struct DropoutKernelArgs {
  const void* x;
  const void* res;
  void* y;
  int64_t n;
  DropMask mask;
  int g_x, g_res, g_y;
};

template <bool BF16, bool STAGED>
__global__ void __launch_bounds__(256) k_dropout(const DropoutKernelArgs a) {
  __shared__ __align__(16) uint8_t stages[STAGED ? 8 : 1][kStageBytes];
  const int lane = threadIdx.x & 31;
  uint8_t* stage = stages[STAGED ? threadIdx.x >> 5 : 0];
  const Dropper drop(a.mask);
  const int64_t step = (int64_t)gridDim.x * 256 * kChunk;
  for (int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * kChunk; e - kChunk * lane < a.n;
       e += step) {
    const int n = chunk_len(e, a.n);
    const int64_t run = warp_run(e - kChunk * lane, a.n);
    ChunkLoad<BF16, STAGED> lx, lr;
    lx.issue(a.x, e, n, run, a.g_x, lane);
    if (a.res != nullptr) lr.issue(a.res, e, n, run, a.g_res, lane);
    float v[kChunk];
    const Chunk<BF16>& cx = lx.settle(a.g_x, stage, lane);
#pragma unroll
    for (int i = 0; i < kChunk; ++i) v[i] = cx.get(i);
    drop.apply(e, v, a.res != nullptr ? &lr.settle(a.g_res, stage, lane) : nullptr);
    Chunk<BF16> cy;
    cy.set(v);
    cy.store_warp<STAGED>(a.y, e, n, run, a.g_y, stage, lane);
  }
}

}  // namespace

cudaError_t launch_dropout(const DropoutArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  if (a.n == 0) return cudaSuccess;
  DropoutKernelArgs k{a.x, a.residual, a.y, a.n, a.mask, row_grain(a.x, 0),
                      row_grain(a.residual, 0), row_grain(a.y, 0)};
  int grain = std::min(k.g_x, k.g_y);
  if (a.residual) grain = std::min(grain, k.g_res);
  const bool bf16 = a.in == InType::BF16;
  // BF16: eight CTAs an SM that walk (what is the call's own is made once, and issue slots are what
  // this is short of beside memory: 134 M elements with a residual 118 us, 131 with a chunk a
  // thread; without one 99 and 115).  FP32 moves twice the bytes for the same instructions and does
  // better without the walk (67 M with a residual 114 us, 123 so).
  const int64_t grid = std::min<int64_t>((a.n + 256 * kChunk - 1) / (256 * kChunk),
                                         bf16 ? 8LL * dev.num_sms : 1 << 20);
  const auto kernel = bf16 ? (grain >= 16 ? k_dropout<true, false> : k_dropout<true, true>)
                           : (grain >= 16 ? k_dropout<false, false> : k_dropout<false, true>);
  kernel<<<(unsigned)grid, 256, 0, stream>>>(k);
  return cudaGetLastError();
}

}  // namespace nvfp4
