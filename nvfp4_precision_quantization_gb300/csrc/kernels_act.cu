// kernels_act.cu -- gradients of bias and activation, with the maxima that the
// quantization of the result needs.
//
//   dz = dd act'(z),  dbias = sum_rows dz,  row_amax / col_amax = max |dz| as stored
//
// Bound by memory (two reads, one write per element).  Sums and maxima over columns and
// rows come out of the same pass, so the quantization that follows reads dz once
// instead of twice.  A warp walks down consecutive rows with 32 bytes of columns per lane
// (16 BF16 or 8 FP32): the column statistics stay in registers, a row's maximum is one warp
// reduction, and a second small kernel joins the partial results in a fixed order (no
// atomics, nothing to clear beforehand).
//
// Measured: 16384 x 28672 BF16 GELU 420 us, 6.7 TB/s, the rate of a copy (769 us with scalar
// arithmetic and without the row loaded ahead; issue slots are now 65 % used); 4000 x 5000
// FP32 SILU 44 us, 5.4 TB/s (a step this short shows its ramp and the joining launch).
#include <algorithm>

#include "activation.cuh"
#include "sector.cuh"

namespace nvfp4 {
namespace {

constexpr int kActThreads = 256;
constexpr int kActWarps = kActThreads / 32;
constexpr int kActMaxCtas = 1024;  // bound of the main kernel's grid, for the workspace

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

template <bool BF16, int ACT, bool STAGED>
__global__ void __launch_bounds__(kActThreads, STAGED ? 2 : 3)
    k_bias_act_backward(const ActKernelArgs a) {
  using S = Sector<BF16>;
  constexpr int kCols = S::kCols, kStrip = 32 * kCols;
  __shared__ float s_sum[kStrip], s_max[kStrip];
  __shared__ __align__(16) uint8_t stages[STAGED ? kActWarps : 1][kStageBytes];
  // the join may be set up meanwhile; without one, the next launch in the stream is another
  // call's, which may count on this one's dz
  if (a.col_sum != nullptr || a.col_max != nullptr || a.row_max != nullptr)
    pdl_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int strip = blockIdx.x % a.strips, part = blockIdx.x / a.strips;
  const int sub = lane / a.lanes, step = 32 / a.lanes;  // rows side by side in the warp
  const int64_t col = (int64_t)strip * kStrip + (lane % a.lanes) * kCols;
  const int n_col = (int)max((int64_t)0, min((int64_t)kCols, a.cols - col));
  // a warp that spans several rows has no run of its own to stage
  uint8_t* stage = STAGED && a.lanes == 32 ? stages[STAGED ? warp : 0] : nullptr;
  const int64_t left = a.cols - (int64_t)strip * kStrip, run = left < kStrip ? left : kStrip;
  // this warp's rows
  const int64_t warps = (int64_t)a.row_parts * kActWarps, w = (int64_t)part * kActWarps + warp;
  const int64_t r0 = a.rows * w / warps, r1 = a.rows * (w + 1) / warps;
  Pair sum[kCols / 2];
  uint32_t mx[8];  // word by word, as dz is stored
#pragma unroll
  for (int i = 0; i < kCols / 2; ++i) sum[i] = {0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < 8; ++i) mx[i] = 0;
  // the next row's words are loaded before this row's are used
  SectorLoad<BF16, STAGED> nd, nz;
  auto fetch = [&](int64_t r) {
    const int n = r < r1 ? n_col : 0;
    const int64_t have = r < r1 ? run : 0;
    nd.issue(a.dd, r * a.cols + col, n, have, a.g_dd, stage, lane);
    if constexpr (ACT != kActNone)
      nz.issue(a.z, r * a.cols + col, n, have, a.g_z, stage, lane);
  };
  fetch(r0 + sub);
  for (int64_t rb = r0; rb < r1; rb += step) {
    const int64_t r = rb + sub;
    S d = nd.settle(a.g_dd, stage, lane), z;
    if constexpr (ACT != kActNone) z = nz.settle(a.g_z, stage, lane);
    if (rb + step < r1) fetch(r + step);
#pragma unroll
    for (int i = 0; i < kCols / 2; ++i) {
      Pair v = d.get(i);
      if constexpr (ACT != kActNone) v = pair_mul(v, act_slope<ACT>(z.get(i)));
      sum[i] = pair_add(sum[i], v);
      d.set(i, v);
    }
    d.store_warp<STAGED>(a.dz, r * a.cols + col, r < r1 ? n_col : 0, r < r1 ? run : 0, a.g_dz, stage, lane);
#pragma unroll
    for (int i = 0; i < 8; ++i) mx[i] = word_absmax<BF16>(mx[i], d.w[i]);
    if (a.row_max != nullptr) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) m = word_absmax<BF16>(m, d.w[i]);
      // as bits: non-negative values are ordered like them
      uint32_t bits = __float_as_uint(word_value<BF16>(m));
      if (a.lanes == 32) {
        bits = __reduce_max_sync(0xffffffffu, bits);
      } else {
        for (int k = a.lanes >> 1; k > 0; k >>= 1)
          bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, k));
      }
      if (r < r1 && lane % a.lanes == 0)
        a.row_max[(int64_t)strip * a.rows + r] = __uint_as_float(bits);
    }
  }
  if (a.col_sum == nullptr && a.col_max == nullptr) return;
  // rows side by side, then the CTA's warps in their order; column c of the strip is kept at
  // (c % kCols) * 32 + c / kCols (no bank conflicts)
  float cmax[kCols], csum[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i) {
    csum[i] = (i & 1) ? sum[i / 2].y : sum[i / 2].x;
    if constexpr (BF16)
      cmax[i] = __uint_as_float(((i & 1) ? mx[i / 2] & 0xffff0000u : mx[i / 2] << 16) & 0x7fffffffu);
    else
      cmax[i] = __uint_as_float(mx[i]);
  }
  for (int k = 16; k >= a.lanes; k >>= 1) {
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
      csum[i] = __fadd_rn(csum[i], __shfl_xor_sync(0xffffffffu, csum[i], k));
      cmax[i] = fmaxf(cmax[i], __shfl_xor_sync(0xffffffffu, cmax[i], k));
    }
  }
  for (int k = 0; k < kActWarps; ++k) {
    if (warp == k && lane < a.lanes) {
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        const int c = i * 32 + lane;
        s_sum[c] = k == 0 ? csum[i] : __fadd_rn(s_sum[c], csum[i]);
        s_max[c] = k == 0 ? cmax[i] : fmaxf(s_max[c], cmax[i]);
      }
    }
    __syncthreads();
  }
  for (int c = threadIdx.x; c < kStrip; c += kActThreads) {
    const int64_t gc = (int64_t)strip * kStrip + c;
    if (gc >= a.cols) break;
    const int at = (c % kCols) * 32 + c / kCols;
    if (a.col_sum != nullptr) a.col_sum[(int64_t)part * a.cols + gc] = s_sum[at];
    if (a.col_max != nullptr) a.col_max[(int64_t)part * a.cols + gc] = s_max[at];
  }
}

int64_t max_row_parts(int64_t cols, bool bf16) {
  return std::max<int64_t>(1, kActMaxCtas / strips_of(cols, bf16));
}

template <bool BF16, int ACT, bool STAGED>
cudaError_t run_act_as(ActKernelArgs& k, const DeviceInfo& dev, cudaStream_t stream) {
  static const int resident = [] {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(
            &n, k_bias_act_backward<BF16, ACT, STAGED>, kActThreads, 0) != cudaSuccess) {
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
  k_bias_act_backward<BF16, ACT, STAGED>
      <<<(unsigned)(k.strips * (int64_t)k.row_parts), kActThreads, 0, stream>>>(k);
  return cudaGetLastError();
}

template <bool BF16, int ACT>
cudaError_t run_act(ActKernelArgs& k, const DeviceInfo& dev, cudaStream_t stream) {
  int grain = std::min(k.g_dd, k.g_dz);
  if (ACT != kActNone) grain = std::min(grain, k.g_z);
  return grain >= 16 ? run_act_as<BF16, ACT, false>(k, dev, stream)
                     : run_act_as<BF16, ACT, true>(k, dev, stream);
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
  // the larger of the two types' needs, part by part
  return 2 * round16(4 * max_row_parts(cols, true) * cols) +
         round16(4 * strips_of(cols, false) * rows);
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
  const bool bf16 = a.in == InType::BF16;
  const int64_t col_bytes = round16(4 * max_row_parts(a.cols, bf16) * a.cols);
  ActKernelArgs k{};
  k.dd = a.dd;
  k.z = a.z;
  k.dz = a.dz;
  k.col_sum = a.dbias ? reinterpret_cast<float*>(ws) : nullptr;
  k.col_max = a.col_amax ? reinterpret_cast<float*>(ws + col_bytes) : nullptr;
  k.row_max = a.row_amax ? reinterpret_cast<float*>(ws + 2 * col_bytes) : nullptr;
  k.rows = a.rows;
  k.cols = a.cols;
  k.strips = (int)strips_of(a.cols, bf16);
  k.lanes = 32;
  while (k.lanes > 1 && (int64_t)(k.lanes / 2) * (bf16 ? 16 : 8) >= a.cols) k.lanes /= 2;
  k.g_dd = row_grain(a.dd, a.cols * e);
  k.g_z = row_grain(a.z, a.cols * e);
  k.g_dz = row_grain(a.dz, a.cols * e);
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
  return launch_after(k_act_join, (unsigned)(r.col_ctas + row_ctas), 256, stream, r);
}

}  // namespace nvfp4
