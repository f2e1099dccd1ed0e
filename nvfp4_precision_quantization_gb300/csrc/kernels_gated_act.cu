// kernels_gated_act.cu -- gradients of d = act(g) u, with the maxima that the quantization of
// the result needs.
//
//   dg = dd u act'(g),  du = dd act(g),  dgu = [dg | du]  (rows of 2 cols values)
//   dbias = sum_rows dgu,  row_amax / col_amax = max |dgu| as stored
//
// Bound by memory (three reads, two writes per element of d).  As in kernels_act.cu a warp
// walks down consecutive rows with 32 bytes of columns per lane, here those of dd and the
// same columns of g and u; act and act' share their exponential and reciprocal.
//
// Measured: 16384 x 14336 BF16 SiLU, sums and maxima 360 us, 6.5 TB/s, 0.96 of a copy; 4000 x 5000
// FP32 GELU 71 us, 5.6 TB/s (ramp and the joining launch).
#include <algorithm>

#include "activation.cuh"
#include "sector.cuh"

namespace nvfp4 {
namespace {

constexpr int kGatedThreads = 256;
constexpr int kGatedWarps = kGatedThreads / 32;
constexpr int kGatedMaxCtas = 1024;  // bound of the main kernel's grid, for the workspace

struct GatedKernelArgs {
  const void* dd;
  const void* gu;
  void* dgu;
  float* col_sum;  // [row_parts][2 cols] or NULL
  float* col_max;  // [row_parts][2 cols] or NULL
  float* row_max;  // [strips][rows] or NULL
  int64_t rows, cols;
  int strips, row_parts;
  int lanes;  // lanes of a warp per row (a power of two): 32 / lanes rows at a time
  int g_dd, g_gu, g_dgu;
};

// Staged BF16 takes half a sector a lane: units of two bytes take a register each, and 32 bytes of
// three tensors beside the sums spill (16000 x 3001 606 us, 146 so).
constexpr __host__ __device__ int sector_words(bool bf16, bool staged) {
  return bf16 && staged ? 4 : 8;
}

template <bool BF16, int ACT, bool STAGED>
__global__ void __launch_bounds__(kGatedThreads, 2) k_gated_backward(const GatedKernelArgs a) {
  constexpr int W = sector_words(BF16, STAGED);
  using S = Sector<BF16, W>;
  constexpr int kCols = S::kCols, kStrip = 32 * kCols;
  __shared__ float s_sum[2][kStrip], s_max[2][kStrip];
  __shared__ __align__(16) uint8_t stages[STAGED ? kGatedWarps : 1][kStageBytes];
  // the join may be set up meanwhile; without one, the next launch in the stream is another
  // call's, which may count on this one's dgu
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
  const int64_t warps = (int64_t)a.row_parts * kGatedWarps, w = (int64_t)part * kGatedWarps + warp;
  const int64_t r0 = a.rows * w / warps, r1 = a.rows * (w + 1) / warps;
  Pair sum[2][kCols / 2];
  uint32_t mx[2][W];  // word by word, as dgu is stored
#pragma unroll
  for (int k = 0; k < 2; ++k) {
#pragma unroll
    for (int i = 0; i < kCols / 2; ++i) sum[k][i] = {0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < W; ++i) mx[k][i] = 0;
  }
  // the next row's words are loaded before this row's are used
  SectorLoad<BF16, STAGED, W> nd, ng, nu;
  auto fetch = [&](int64_t r) {
    const int n = r < r1 ? n_col : 0;
    const int64_t have = r < r1 ? run : 0;
    nd.issue(a.dd, r * a.cols + col, n, have, a.g_dd, stage, lane);
    ng.issue(a.gu, 2 * r * a.cols + col, n, have, a.g_gu, stage, lane);
    nu.issue(a.gu, (2 * r + 1) * a.cols + col, n, have, a.g_gu, stage, lane);
  };
  fetch(r0 + sub);
  for (int64_t rb = r0; rb < r1; rb += step) {
    const int64_t r = rb + sub;
    const S d = nd.settle(a.g_dd, stage, lane);
    S g = ng.settle(a.g_gu, stage, lane);
    S u = nu.settle(a.g_gu, stage, lane);
    if (rb + step < r1) fetch(r + step);
#pragma unroll
    for (int i = 0; i < kCols / 2; ++i) {
      const Pair dd = d.get(i);
      Pair value;
      const Pair slope = act_slope<ACT>(g.get(i), value);
      Pair dg = pair_mul(dd, u.get(i));
      if constexpr (ACT != kActNone) dg = pair_mul(dg, slope);
      const Pair du = pair_mul(dd, value);
      sum[0][i] = pair_add(sum[0][i], dg);
      sum[1][i] = pair_add(sum[1][i], du);
      g.set(i, dg);
      u.set(i, du);
    }
    const int n = r < r1 ? n_col : 0;
    const int64_t have = r < r1 ? run : 0;
    g.template store_warp<STAGED>(a.dgu, 2 * r * a.cols + col, n, have, a.g_dgu, stage, lane);
    u.template store_warp<STAGED>(a.dgu, (2 * r + 1) * a.cols + col, n, have, a.g_dgu, stage, lane);
#pragma unroll
    for (int i = 0; i < W; ++i) {
      mx[0][i] = word_absmax<BF16>(mx[0][i], g.w[i]);
      mx[1][i] = word_absmax<BF16>(mx[1][i], u.w[i]);
    }
    if (a.row_max != nullptr) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < W; ++i) m = word_absmax<BF16>(word_absmax<BF16>(m, g.w[i]), u.w[i]);
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
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float cmax[kCols], csum[kCols];
#pragma unroll
    for (int i = 0; i < kCols; ++i) {
      csum[i] = (i & 1) ? sum[h][i / 2].y : sum[h][i / 2].x;
      if constexpr (BF16)
        cmax[i] = __uint_as_float(
            ((i & 1) ? mx[h][i / 2] & 0xffff0000u : mx[h][i / 2] << 16) & 0x7fffffffu);
      else
        cmax[i] = __uint_as_float(mx[h][i]);
    }
    for (int k = 16; k >= a.lanes; k >>= 1) {
#pragma unroll
      for (int i = 0; i < kCols; ++i) {
        csum[i] = __fadd_rn(csum[i], __shfl_xor_sync(0xffffffffu, csum[i], k));
        cmax[i] = fmaxf(cmax[i], __shfl_xor_sync(0xffffffffu, cmax[i], k));
      }
    }
    for (int k = 0; k < kGatedWarps; ++k) {
      if (warp == k && lane < a.lanes) {
#pragma unroll
        for (int i = 0; i < kCols; ++i) {
          const int c = i * 32 + lane;
          s_sum[h][c] = k == 0 ? csum[i] : __fadd_rn(s_sum[h][c], csum[i]);
          s_max[h][c] = k == 0 ? cmax[i] : fmaxf(s_max[h][c], cmax[i]);
        }
      }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < kStrip; c += kGatedThreads) {
      const int64_t gc = (int64_t)strip * kStrip + c;
      if (gc >= a.cols) break;
      const int at = (c % kCols) * 32 + c / kCols;
      const int64_t to = ((int64_t)part * 2 + h) * a.cols + gc;
      if (a.col_sum != nullptr) a.col_sum[to] = s_sum[h][at];
      if (a.col_max != nullptr) a.col_max[to] = s_max[h][at];
    }
  }
}

int64_t max_row_parts(int64_t cols, bool bf16) {
  return std::max<int64_t>(1, kGatedMaxCtas / strips_of(cols, bf16));
}

// Whether some tensor's rows do not allow 16-byte accesses.
bool staged(const GatedKernelArgs& k) {
  return std::min(k.g_dd, std::min(k.g_gu, k.g_dgu)) < 16;
}

template <bool BF16, int ACT, bool STAGED>
cudaError_t run_as(GatedKernelArgs& k, const DeviceInfo& dev, cudaStream_t stream) {
  static const int resident = [] {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, k_gated_backward<BF16, ACT, STAGED>,
                                                      kGatedThreads, 0) != cudaSuccess) {
      cudaGetLastError();
      n = 2;
    }
    return std::max(1, n);
  }();
  // one wave of CTAs, each warp at least one group of rows
  const int64_t fill = std::min<int64_t>((int64_t)resident * dev.num_sms, kGatedMaxCtas);
  const int64_t rows_per_cta = (int64_t)kGatedWarps * (32 / k.lanes);
  k.row_parts = (int)std::max<int64_t>(
      1, std::min(fill / k.strips, (k.rows + rows_per_cta - 1) / rows_per_cta));
  k_gated_backward<BF16, ACT, STAGED>
      <<<(unsigned)(k.strips * (int64_t)k.row_parts), kGatedThreads, 0, stream>>>(k);
  return cudaGetLastError();
}

template <bool BF16, int ACT>
cudaError_t run(GatedKernelArgs& k, const DeviceInfo& dev, cudaStream_t stream) {
  return staged(k) ? run_as<BF16, ACT, true>(k, dev, stream)
                   : run_as<BF16, ACT, false>(k, dev, stream);
}

template <bool BF16>
cudaError_t pick(int act, GatedKernelArgs& k, const DeviceInfo& dev, cudaStream_t stream) {
  switch (act) {
    case kActRelu: return run<BF16, kActRelu>(k, dev, stream);
    case kActGelu: return run<BF16, kActGelu>(k, dev, stream);
    case kActSilu: return run<BF16, kActSilu>(k, dev, stream);
    default: return run<BF16, kActNone>(k, dev, stream);
  }
}

}  // namespace

int64_t gated_backward_workspace(int64_t rows, int64_t cols) {
  // the larger of the two types' needs, part by part
  return 2 * round16(8 * max_row_parts(cols, true) * cols) +
         round16(4 * strips_of(cols, false) * rows);
}

cudaError_t launch_gated_backward(const GatedBackwardArgs& a, const DeviceInfo& dev,
                                  cudaStream_t stream) {
  if (a.rows == 0 || a.cols == 0) {  // empty sums and maxima
    cudaError_t e = cudaSuccess;
    if (a.dbias && a.cols) e = cudaMemsetAsync(a.dbias, 0, 8 * a.cols, stream);
    if (e == cudaSuccess && a.col_amax && a.cols)
      e = cudaMemsetAsync(a.col_amax, 0, 8 * a.cols, stream);
    if (e == cudaSuccess && a.row_amax && a.rows)
      e = cudaMemsetAsync(a.row_amax, 0, 4 * a.rows, stream);
    return e;
  }
  const bool bf16 = a.in == InType::BF16;
  const int e = bf16 ? 2 : 4;
  char* ws = static_cast<char*>(a.workspace);
  const int64_t col_bytes = round16(8 * max_row_parts(a.cols, bf16) * a.cols);
  GatedKernelArgs k{};
  k.dd = a.dd;
  k.gu = a.gu;
  k.dgu = a.dgu;
  k.col_sum = a.dbias ? reinterpret_cast<float*>(ws) : nullptr;
  k.col_max = a.col_amax ? reinterpret_cast<float*>(ws + col_bytes) : nullptr;
  k.row_max = a.row_amax ? reinterpret_cast<float*>(ws + 2 * col_bytes) : nullptr;
  k.rows = a.rows;
  k.cols = a.cols;
  k.g_dd = row_grain(a.dd, a.cols * e);
  k.g_gu = row_grain(a.gu, a.cols * e);  // u starts `cols` into the row
  k.g_dgu = row_grain(a.dgu, a.cols * e);
  const int words = sector_words(bf16, staged(k)), lane_cols = bf16 ? 2 * words : words;
  k.strips = (int)strips_of(a.cols, bf16, words == 4);
  k.lanes = 32;
  while (k.lanes > 1 && (int64_t)(k.lanes / 2) * lane_cols >= a.cols) k.lanes /= 2;
  cudaError_t err = bf16 ? pick<true>(a.act, k, dev, stream) : pick<false>(a.act, k, dev, stream);
  if (err != cudaSuccess || !(a.dbias || a.col_amax || a.row_amax)) return err;
  ActReduceArgs r{};
  r.col_sum = k.col_sum;
  r.col_max = k.col_max;
  r.row_max = k.row_max;
  r.dbias = a.dbias;
  r.col_amax = a.col_amax;
  r.row_amax = a.row_amax;
  r.rows = a.rows;
  r.cols = 2 * a.cols;
  r.strips = k.strips;
  r.row_parts = k.row_parts;
  r.col_ctas = a.dbias || a.col_amax ? (int)((2 * a.cols + 31) / 32) : 0;
  const int64_t row_ctas = a.row_amax ? (a.rows + 255) / 256 : 0;
  return launch_after(k_act_join, (unsigned)(r.col_ctas + row_ctas), 256, stream, r);
}

}  // namespace nvfp4
