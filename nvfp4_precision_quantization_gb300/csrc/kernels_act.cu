// kernels_act.cu -- gradients of bias and activation, with the maxima that the
// quantization of the result needs.
//
//   dz = dd act'(z),  dbias = sum_rows dz,  row_amax / col_amax = max |dz| as stored
//
// Bound by memory (two reads, one write per element).  Sums and maxima over columns and
// rows come out of the same pass, so the quantization that follows reads dz once
// instead of twice.  A warp walks down consecutive rows with 16 columns per lane: the
// column statistics stay in registers, a row's maximum is one warp reduction, and a
// second small kernel joins the partial results in a fixed order (no atomics, nothing to
// clear beforehand).
#include <algorithm>

#include "activation.cuh"
#include "internal.h"
#include "row_io.cuh"

namespace nvfp4 {
namespace {

constexpr int kActThreads = 256;
constexpr int kActWarps = kActThreads / 32;
constexpr int kActMaxCtas = 1024;  // bound of the main kernel's grid, for the workspace
constexpr int kStrip = 32 * kChunk;  // columns of one warp

struct ActKernelArgs {
  const void* dd;
  const void* z;
  void* dz;
  float* col_sum;  // [row_parts][cols] or NULL
  float* col_max;  // [row_parts][cols] or NULL
  float* row_max;  // [strips][rows] or NULL
  int64_t rows, cols;
  int strips, row_parts;
  int lanes;  // lanes of a warp per row (a power of two): 32 / lanes rows at a time
  int g_dd, g_z, g_dz;
};

template <bool BF16, int ACT>
__global__ void __launch_bounds__(kActThreads, 2) k_bias_act_backward(const ActKernelArgs a) {
  __shared__ float s_sum[kStrip], s_max[kStrip];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int strip = blockIdx.x % a.strips, part = blockIdx.x / a.strips;
  const int sub = lane / a.lanes, step = 32 / a.lanes;  // rows side by side in the warp
  const int64_t col = (int64_t)strip * kStrip + (lane % a.lanes) * kChunk;
  const int n_col = chunk_len(col, a.cols);
  // this warp's rows
  const int64_t warps = (int64_t)a.row_parts * kActWarps, w = (int64_t)part * kActWarps + warp;
  const int64_t r0 = a.rows * w / warps, r1 = a.rows * (w + 1) / warps;
  float sum[kChunk], mx[kChunk];
#pragma unroll
  for (int i = 0; i < kChunk; ++i) sum[i] = mx[i] = 0.0f;
  for (int64_t rb = r0; rb < r1; rb += step) {
    const int64_t r = rb + sub;
    const int n = r < r1 ? n_col : 0;
    const int64_t off = r * a.cols + col;
    Chunk<BF16> cd, cz;
    cd.load(a.dd, off, n, a.g_dd);
    if constexpr (ACT != kActNone) cz.load(a.z, off, n, a.g_z);
    float v[kChunk];
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      v[i] = cd.get(i);
      if constexpr (ACT != kActNone) v[i] = __fmul_rn(v[i], act_slope<ACT>(cz.get(i)));
      sum[i] = __fadd_rn(sum[i], v[i]);
    }
    cd.set(v);
    cd.store(a.dz, off, n, a.g_dz);
    float rm = 0.0f;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      const float m = fabsf(cd.get(i));
      mx[i] = fmaxf(mx[i], m);
      rm = fmaxf(rm, m);
    }
    if (a.row_max != nullptr) {
      for (int d = a.lanes >> 1; d > 0; d >>= 1)
        rm = fmaxf(rm, __shfl_xor_sync(0xffffffffu, rm, d));
      if (r < r1 && lane % a.lanes == 0) a.row_max[(int64_t)strip * a.rows + r] = rm;
    }
  }
  if (a.col_sum == nullptr && a.col_max == nullptr) return;
  // rows side by side, then the CTA's warps in their order
  for (int d = 16; d >= a.lanes; d >>= 1) {
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      sum[i] = __fadd_rn(sum[i], __shfl_xor_sync(0xffffffffu, sum[i], d));
      mx[i] = fmaxf(mx[i], __shfl_xor_sync(0xffffffffu, mx[i], d));
    }
  }
  for (int k = 0; k < kActWarps; ++k) {
    if (warp == k && lane < a.lanes) {
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        const int c = i * 32 + lane;  // lane-major columns: no bank conflicts
        s_sum[c] = k == 0 ? sum[i] : __fadd_rn(s_sum[c], sum[i]);
        s_max[c] = k == 0 ? mx[i] : fmaxf(s_max[c], mx[i]);
      }
    }
    __syncthreads();
  }
  for (int c = threadIdx.x; c < kStrip; c += kActThreads) {
    const int64_t gc = (int64_t)strip * kStrip + c;
    if (gc >= a.cols) break;
    const int at = (c % kChunk) * 32 + c / kChunk;
    if (a.col_sum != nullptr) a.col_sum[(int64_t)part * a.cols + gc] = s_sum[at];
    if (a.col_max != nullptr) a.col_max[(int64_t)part * a.cols + gc] = s_max[at];
  }
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
  if ((int)blockIdx.x < a.col_ctas) {
    __shared__ float s_sum[8][32], s_max[8][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float sum = 0.0f, mx = 0.0f;
    if (c < a.cols) {
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
    for (int s = 0; s < a.strips; ++s) mx = fmaxf(mx, a.row_max[(int64_t)s * a.rows + r]);
    a.row_amax[r] = mx;
  }
}

int64_t strips_of(int64_t cols) { return (cols + kStrip - 1) / kStrip; }
int64_t max_row_parts(int64_t cols) {
  return std::max<int64_t>(1, kActMaxCtas / strips_of(cols));
}
int64_t round16(int64_t v) { return (v + 15) / 16 * 16; }

template <bool BF16, int ACT>
cudaError_t run_act(ActKernelArgs& k, const DeviceInfo& dev, cudaStream_t stream) {
  static const int resident = [] {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k_bias_act_backward<BF16, ACT>,
                                                      kActThreads, 0) != cudaSuccess) {
      cudaGetLastError();
      n = 2;
    }
    return std::max(1, n);
  }();
  // one wave of CTAs, each warp at least one group of rows
  const int64_t fill = std::min<int64_t>((int64_t)resident * dev.num_sms, kActMaxCtas);
  const int64_t rows_per_cta = (int64_t)kActWarps * (32 / k.lanes);
  k.row_parts = (int)std::max<int64_t>(
      1, std::min(fill / k.strips, (k.rows + rows_per_cta - 1) / rows_per_cta));
  k_bias_act_backward<BF16, ACT>
      <<<(unsigned)(k.strips * (int64_t)k.row_parts), kActThreads, 0, stream>>>(k);
  return cudaGetLastError();
}

template <bool BF16>
cudaError_t pick_act(int act, ActKernelArgs& k, const DeviceInfo& dev, cudaStream_t stream) {
  switch (act) {
    case kActRelu: return run_act<BF16, kActRelu>(k, dev, stream);
    case kActGelu: return run_act<BF16, kActGelu>(k, dev, stream);
    case kActSilu: return run_act<BF16, kActSilu>(k, dev, stream);
    default: return run_act<BF16, kActNone>(k, dev, stream);
  }
}

}  // namespace

int64_t bias_act_backward_workspace(int64_t rows, int64_t cols) {
  return 2 * round16(4 * max_row_parts(cols) * cols) + round16(4 * strips_of(cols) * rows);
}

cudaError_t launch_bias_act_backward(const ActBackwardArgs& a, const DeviceInfo& dev,
                                     cudaStream_t stream) {
  if (a.rows == 0 || a.cols == 0) {  // empty sums and maxima
    cudaError_t e = cudaSuccess;
    if (a.dbias && a.cols) e = cudaMemsetAsync(a.dbias, 0, 4 * a.cols, stream);
    if (e == cudaSuccess && a.col_amax && a.cols)
      e = cudaMemsetAsync(a.col_amax, 0, 4 * a.cols, stream);
    if (e == cudaSuccess && a.row_amax && a.rows)
      e = cudaMemsetAsync(a.row_amax, 0, 4 * a.rows, stream);
    return e;
  }
  const int e = a.in == InType::BF16 ? 2 : 4;
  char* ws = static_cast<char*>(a.workspace);
  const int64_t col_bytes = round16(4 * max_row_parts(a.cols) * a.cols);
  ActKernelArgs k{};
  k.dd = a.dd;
  k.z = a.z;
  k.dz = a.dz;
  k.col_sum = a.dbias ? reinterpret_cast<float*>(ws) : nullptr;
  k.col_max = a.col_amax ? reinterpret_cast<float*>(ws + col_bytes) : nullptr;
  k.row_max = a.row_amax ? reinterpret_cast<float*>(ws + 2 * col_bytes) : nullptr;
  k.rows = a.rows;
  k.cols = a.cols;
  k.strips = (int)strips_of(a.cols);
  k.lanes = 32;
  while (k.lanes > 1 && (int64_t)(k.lanes / 2) * kChunk >= a.cols) k.lanes /= 2;
  k.g_dd = row_grain(a.dd, a.cols, e);
  k.g_z = row_grain(a.z, a.cols, e);
  k.g_dz = row_grain(a.dz, a.cols, e);
  cudaError_t err = a.in == InType::BF16 ? pick_act<true>(a.act, k, dev, stream)
                                         : pick_act<false>(a.act, k, dev, stream);
  if (err != cudaSuccess || !(a.dbias || a.col_amax || a.row_amax)) return err;
  ActReduceArgs r{};
  r.col_sum = k.col_sum;
  r.col_max = k.col_max;
  r.row_max = k.row_max;
  r.dbias = a.dbias;
  r.col_amax = a.col_amax;
  r.row_amax = a.row_amax;
  r.rows = a.rows;
  r.cols = a.cols;
  r.strips = k.strips;
  r.row_parts = k.row_parts;
  r.col_ctas = a.dbias || a.col_amax ? (int)((a.cols + 31) / 32) : 0;
  const int64_t row_ctas = a.row_amax ? (a.rows + 255) / 256 : 0;
  k_act_join<<<(unsigned)(r.col_ctas + row_ctas), 256, 0, stream>>>(r);
  return cudaGetLastError();
}

}  // namespace nvfp4
