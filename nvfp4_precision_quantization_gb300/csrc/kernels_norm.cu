// kernels_norm.cu -- residual addition and root-mean-square norm with a quantized
// output, and its gradients.
//
//   h = x + residual,  s = 1 / sqrt(mean(h^2) + eps),  y = h * w * s
//   dx = s (g - n mean(g n)) + dh,  dw = sum_rows dy n,   n = h s,  g = dy w
//
// Both are bound by memory: every tensor is read or written once.  A row's team of
// threads holds the row in registers (16 consecutive elements per thread and step), so
// neither the statistic nor the row's amax needs a second read.  The forward takes both
// in one reduction: amax(y) = s max|h w| exactly, because rounding after the product
// with the positive s is monotonic; the scale of the whole row is therefore known one
// barrier after its last load.
#include <algorithm>

#include "internal.h"
#include "row_io.cuh"

namespace nvfp4 {
namespace {

struct NormKernelArgs {
  const void* x;
  const void* res;
  const void* w;
  void* h;
  void* y;
  float* rstd;
  uint8_t* q8;
  float* q8_scale;
  bool q8_blocks;  // a scale per 128 columns instead of per row
  uint8_t* codes;
  uint8_t* scales;
  float* amax;
  const float* amax_in;
  bool amax_per_tensor;
  bool four_over_six;
  float F, F_inv, negz;
  int64_t rows;
  int cols;
  float eps;
  bool w_bf16;
  int g_x, g_res, g_w, g_h, g_y;  // row grains (row_io.cuh)
};

constexpr float kE4m3Max = 448.0f;

// Encode scale of an E4M3 output whose largest magnitude is a.
__device__ __forceinline__ float fp8_encode_scale(float a) { return global_scale(a, kE4m3Max); }
__device__ __forceinline__ float fp8_decode_scale(float a) {
  return a == 0.0f ? 1.0f : fmaxf(__fdiv_rn(a, kE4m3Max), 0x1p-126f);
}

// Sum and maximum over the TPR threads of a row's team; every thread gets both.  The
// order of the sum depends on TPR alone.  red: two buffers of one pair per warp, used in
// turn, so that one barrier per row is enough.
template <int TPR>
__device__ __forceinline__ float2 team_sum_max(float s, float m, float2* red) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, d));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  }
  if constexpr (TPR > 32) {
    const int warp = threadIdx.x >> 5, first = warp - warp % (TPR / 32);
    if ((threadIdx.x & 31) == 0) red[warp] = make_float2(s, m);
    __syncthreads();
    s = 0.0f;
    m = 0.0f;
#pragma unroll
    for (int i = 0; i < TPR / 32; ++i) {
      const float2 v = red[first + i];
      s = __fadd_rn(s, v.x);
      m = fmaxf(m, v.y);
    }
  }
  return make_float2(s, m);
}

template <bool BF16, bool NV4, int TPR, int NCH>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) k_add_rmsnorm(const NormKernelArgs a) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  constexpr int kTeams = kThreads / TPR;
  __shared__ float2 red[2][kThreads / 32];
  const int t = threadIdx.x % TPR, team = threadIdx.x / TPR;
  int buf = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * kTeams; row0 < a.rows;
       row0 += (int64_t)gridDim.x * kTeams, buf ^= 1) {
    const int64_t row = row0 + team;
    const bool live = row < a.rows;
    const int64_t base = row * a.cols;
    float v[NCH][kChunk];  // h, then h w, then y
    float ss = 0.0f, mx = 0.0f;
    float bmax[NCH];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int col = (c * TPR + t) * kChunk;
      const int n = live ? chunk_len(col, a.cols) : 0;
      Chunk<BF16> cx;
      cx.load(a.x, base + col, n, a.g_x);
#pragma unroll
      for (int i = 0; i < kChunk; ++i) v[c][i] = cx.get(i);
      if (a.res != nullptr) {
        Chunk<BF16> cr;
        cr.load(a.res, base + col, n, a.g_res);
#pragma unroll
        for (int i = 0; i < kChunk; ++i) v[c][i] = __fadd_rn(v[c][i], cr.get(i));
      }
    }
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int col = (c * TPR + t) * kChunk;
      const int n = live ? chunk_len(col, a.cols) : 0;
      if (a.h != nullptr) {
        Chunk<BF16> ch;
        ch.set(v[c]);
        ch.store(a.h, base + col, n, a.g_h);
      }
      float w[kChunk];
      load_vector16(a.w, a.w_bf16, col, n, a.g_w, w);
      float b = 0.0f;
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        ss = __fmaf_rn(v[c][i], v[c][i], ss);
        v[c][i] = __fmul_rn(v[c][i], w[i]);
        b = fmaxf(b, fabsf(v[c][i]));
      }
      bmax[c] = b;
      mx = fmaxf(mx, b);
    }
    const float2 r = team_sum_max<TPR>(ss, mx, red[buf]);
    const float mean = a.cols > 0 ? __fdiv_rn(r.x, (float)a.cols) : 0.0f;
    const float s = __frsqrt_rn(__fadd_rn(mean, a.eps));
    const float top = __fmul_rn(r.y, s);  // amax of the row's y
    if (live && t == 0 && a.rstd != nullptr) a.rstd[row] = s;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int i = 0; i < kChunk; ++i) v[c][i] = __fmul_rn(v[c][i], s);
    if (a.y != nullptr) {
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int col = (c * TPR + t) * kChunk;
        Chunk<BF16> cy;
        cy.set(v[c]);
        cy.store(a.y, base + col, live ? chunk_len(col, a.cols) : 0, a.g_y);
      }
    }
    if constexpr (NV4) {
      float line = top;
      if (a.amax_in != nullptr && live) line = a.amax_in[a.amax_per_tensor ? 0 : row];
      if (live && t == 0 && (!a.amax_per_tensor || row == 0) && a.amax != a.amax_in)
        a.amax[a.amax_per_tensor ? 0 : row] = line;
      const float S = global_scale(line, a.F);
      const int64_t cpitch = (a.cols + 1) / 2, spitch = (a.cols + 15) / 16;
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int col = (c * TPR + t) * kChunk;
        const int n = live ? chunk_len(col, a.cols) : 0;
        if (n == 0) continue;
        const float b = __fmul_rn(bmax[c], s);
        uint32_t cw[2];
        uint32_t s8;
        if (a.four_over_six)
          s8 = quantize16<true>(v[c], b, S, line, a.F_inv, a.negz, cw[0], cw[1]);
        else
          s8 = quantize16<false>(v[c], b, S, line, a.F_inv, a.negz, cw[0], cw[1]);
        store_bytes(a.codes + row * cpitch + col / 2, cw, (n + 1) / 2);
        a.scales[row * spitch + col / 16] = (uint8_t)s8;
      }
    } else if (a.q8 != nullptr) {
      if (live && t == 0 && !a.q8_blocks) a.q8_scale[row] = fp8_decode_scale(top);
      const float S_row = fp8_encode_scale(top);
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int col = (c * TPR + t) * kChunk;
        const int n = live ? chunk_len(col, a.cols) : 0;
        float S = S_row;
        if (a.q8_blocks) {  // 128 columns are eight neighbouring lanes
          float b = bmax[c];
#pragma unroll
          for (int d = 4; d > 0; d >>= 1) b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, d));
          b = __fmul_rn(b, s);
          S = fp8_encode_scale(b);
          if (n > 0 && (t & 7) == 0)
            a.q8_scale[row * ((a.cols + 127) / 128) + col / 128] = fp8_decode_scale(b);
        }
        if (n == 0) continue;
        uint32_t cw[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint16_t lo, hi;
          asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
              : "=h"(lo)
              : "f"(__fmul_rn(v[c][4 * i + 1], S)), "f"(__fmul_rn(v[c][4 * i], S)));
          asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
              : "=h"(hi)
              : "f"(__fmul_rn(v[c][4 * i + 3], S)), "f"(__fmul_rn(v[c][4 * i + 2], S)));
          cw[i] = (uint32_t)lo | ((uint32_t)hi << 16);
        }
        store_bytes(a.q8 + base + col, cw, n);
      }
    }
  }
}

// ---------------------------------------------------------------- backward

struct NormBackwardKernelArgs {
  const void* dy;
  const void* h;
  const void* dh;
  const void* w;
  const float* rstd;
  void* dx;
  float* part;  // [gridDim.x][cols] partial dweight, or NULL
  int64_t rows;
  int cols;
  bool w_bf16;
  int g_dy, g_h, g_dh, g_w, g_dx;
};

// CTA b takes the rows b, b + gridDim.x, ... (times its teams); each thread keeps the
// weight's gradient of its own columns in registers over all of them, so dw costs one
// row of partial sums per CTA.
template <bool BF16, int TPR, int NCH>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
    k_add_rmsnorm_backward(const NormBackwardKernelArgs a) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  constexpr int kTeams = kThreads / TPR;
  __shared__ float2 red[2][kThreads / 32];
  __shared__ float s_dw[kTeams > 1 ? TPR * NCH * kChunk : 1];
  const int t = threadIdx.x % TPR, team = threadIdx.x / TPR;
  float dw[NCH][kChunk];
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int i = 0; i < kChunk; ++i) dw[c][i] = 0.0f;
  int buf = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * kTeams; row0 < a.rows;
       row0 += (int64_t)gridDim.x * kTeams, buf ^= 1) {
    const int64_t row = row0 + team;
    const bool live = row < a.rows;
    const int64_t base = row * a.cols;
    const float s = live ? a.rstd[row] : 0.0f;
    Chunk<BF16> cy[NCH], ch[NCH];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int col = (c * TPR + t) * kChunk;
      const int n = live ? chunk_len(col, a.cols) : 0;
      cy[c].load(a.dy, base + col, n, a.g_dy);
      ch[c].load(a.h, base + col, n, a.g_h);
    }
    float dot = 0.0f;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int col = (c * TPR + t) * kChunk;
      float w[kChunk];
      load_vector16(a.w, a.w_bf16, col, chunk_len(col, a.cols), a.g_w, w);
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        const float dyn = __fmul_rn(cy[c].get(i), __fmul_rn(ch[c].get(i), s));
        dw[c][i] = __fadd_rn(dw[c][i], dyn);
        dot = __fmaf_rn(dyn, w[i], dot);
      }
    }
    const float2 r = team_sum_max<TPR>(dot, 0.0f, red[buf]);
    const float mean = __fdiv_rn(r.x, (float)a.cols);
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int col = (c * TPR + t) * kChunk;
      const int n = live ? chunk_len(col, a.cols) : 0;
      float w[kChunk], dx[kChunk];
      load_vector16(a.w, a.w_bf16, col, chunk_len(col, a.cols), a.g_w, w);
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        const float g = __fmul_rn(cy[c].get(i), w[i]);
        const float nn = __fmul_rn(ch[c].get(i), s);
        dx[i] = __fmul_rn(__fmaf_rn(-nn, mean, g), s);
      }
      if (a.dh != nullptr) {
        Chunk<BF16> cd;
        cd.load(a.dh, base + col, n, a.g_dh);
#pragma unroll
        for (int i = 0; i < kChunk; ++i) dx[i] = __fadd_rn(dx[i], cd.get(i));
      }
      Chunk<BF16> co;
      co.set(dx);
      co.store(a.dx, base + col, n, a.g_dx);
    }
  }
  if (a.part == nullptr) return;
  if constexpr (kTeams > 1) {  // the CTA's teams in their order
    for (int k = 0; k < kTeams; ++k) {
      if (team == k) {
#pragma unroll
        for (int c = 0; c < NCH; ++c)
#pragma unroll
          for (int i = 0; i < kChunk; ++i) {
            float* p = &s_dw[(c * TPR + t) * kChunk + i];
            *p = k == 0 ? dw[c][i] : __fadd_rn(*p, dw[c][i]);
          }
      }
      __syncthreads();
    }
    for (int i = threadIdx.x; i < a.cols; i += kThreads)
      a.part[(int64_t)blockIdx.x * a.cols + i] = s_dw[i];
  } else {
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int col = (c * TPR + t) * kChunk;
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        if (col + i < a.cols) a.part[(int64_t)blockIdx.x * a.cols + col + i] = dw[c][i];
    }
  }
}

// out[c] = sum over the n partial rows of part [n][cols], in a fixed order: warp w of a
// CTA adds the rows w, w + 8, ..., and the eight sums are added in turn.
__global__ void __launch_bounds__(256) k_column_sum(const float* part, int n, int64_t cols,
                                                    float* out) {
  __shared__ float s[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  float sum = 0.0f;
  if (col < cols)
    for (int r = warp; r < n; r += 8) sum = __fadd_rn(sum, part[(int64_t)r * cols + col]);
  s[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && col < cols) {
#pragma unroll
    for (int i = 1; i < 8; ++i) sum = __fadd_rn(sum, s[i][lane]);
    out[col] = sum;
  }
}

template <typename K>
int resident_ctas(K kernel, int threads) {
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0) != cudaSuccess) {
    cudaGetLastError();
    n = 1;
  }
  return std::max(1, n);
}

template <bool BF16, bool NV4, int TPR, int NCH>
cudaError_t run_norm(const NormKernelArgs& k, const DeviceInfo& dev, cudaStream_t stream) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  static const int resident = resident_ctas(k_add_rmsnorm<BF16, NV4, TPR, NCH>, kThreads);
  const int64_t groups = (k.rows + kThreads / TPR - 1) / (kThreads / TPR);
  const int64_t grid = std::min<int64_t>(groups, (int64_t)resident * dev.num_sms);
  k_add_rmsnorm<BF16, NV4, TPR, NCH><<<(unsigned)grid, kThreads, 0, stream>>>(k);
  return cudaGetLastError();
}

template <bool BF16, bool NV4>
cudaError_t pick_norm(const NormKernelArgs& k, const DeviceInfo& dev, cudaStream_t stream) {
  // one step of 16 elements per thread while the rows do not fill the GPU, two beyond
  const bool few = k.rows <= 2LL * dev.num_sms;
  const int c = k.cols;
  if (c <= 512) return run_norm<BF16, NV4, 32, 1>(k, dev, stream);
  if (c <= 1024 && !few) return run_norm<BF16, NV4, 32, 2>(k, dev, stream);
  if (c <= 2048) return run_norm<BF16, NV4, 128, 1>(k, dev, stream);
  if (c <= 4096) return run_norm<BF16, NV4, 256, 1>(k, dev, stream);
  if (c <= 8192 && !few) return run_norm<BF16, NV4, 256, 2>(k, dev, stream);
  if (c <= 8192) return run_norm<BF16, NV4, 512, 1>(k, dev, stream);
  if (c <= 16384 && !few) return run_norm<BF16, NV4, 512, 2>(k, dev, stream);
  if (c <= 16384) return run_norm<BF16, NV4, 1024, 1>(k, dev, stream);
  return run_norm<BF16, NV4, 1024, 2>(k, dev, stream);
}

template <bool BF16, int TPR, int NCH>
cudaError_t run_norm_backward(const NormBackwardKernelArgs& k, int max_parts,
                              const DeviceInfo& dev, cudaStream_t stream, int* parts) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  static const int resident = resident_ctas(k_add_rmsnorm_backward<BF16, TPR, NCH>, kThreads);
  const int64_t groups = (k.rows + kThreads / TPR - 1) / (kThreads / TPR);
  const int grid = (int)std::min<int64_t>(
      std::min<int64_t>(groups, (int64_t)resident * dev.num_sms), max_parts);
  *parts = grid;
  k_add_rmsnorm_backward<BF16, TPR, NCH><<<grid, kThreads, 0, stream>>>(k);
  return cudaGetLastError();
}

template <bool BF16>
cudaError_t pick_norm_backward(const NormBackwardKernelArgs& k, int max_parts,
                               const DeviceInfo& dev, cudaStream_t stream, int* parts) {
  const int c = k.cols;
  if (c <= 512) return run_norm_backward<BF16, 32, 1>(k, max_parts, dev, stream, parts);
  if (c <= 2048) return run_norm_backward<BF16, 128, 1>(k, max_parts, dev, stream, parts);
  if (c <= 4096) return run_norm_backward<BF16, 256, 1>(k, max_parts, dev, stream, parts);
  if (c <= 8192) return run_norm_backward<BF16, 512, 1>(k, max_parts, dev, stream, parts);
  if (c <= 16384) return run_norm_backward<BF16, 1024, 1>(k, max_parts, dev, stream, parts);
  return run_norm_backward<BF16, 1024, 2>(k, max_parts, dev, stream, parts);
}

}  // namespace

cudaError_t launch_column_sum(const float* part, int n, int64_t cols, float* out,
                              cudaStream_t stream) {
  k_column_sum<<<(unsigned)((cols + 31) / 32), 256, 0, stream>>>(part, n, cols, out);
  return cudaGetLastError();
}

cudaError_t launch_add_rmsnorm(const NormArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  if (a.rows == 0) return cudaSuccess;
  const int e = a.in == InType::BF16 ? 2 : 4;
  NormKernelArgs k{};
  k.x = a.x;
  k.res = a.residual;
  k.w = a.weight;
  k.h = a.h;
  k.y = a.y;
  k.rstd = a.rstd;
  k.q8 = a.q8;
  k.q8_scale = a.q8_scale;
  k.q8_blocks = a.q8_block != 0;
  k.codes = a.codes;
  k.scales = a.scales;
  k.amax = a.amax;
  k.amax_in = a.amax_in;
  k.amax_per_tensor = a.amax_per_tensor;
  k.four_over_six = a.four_over_six;
  k.F = a.bound * 6.0f;
  k.F_inv = 1.0f / (a.bound * 6.0f);
  k.negz = -0.0f;
  k.rows = a.rows;
  k.cols = (int)a.cols;
  k.eps = a.eps;
  k.w_bf16 = a.weight_bf16;
  k.g_x = row_grain(a.x, a.cols, e);
  k.g_res = row_grain(a.residual, a.cols, e);
  k.g_h = row_grain(a.h, a.cols, e);
  k.g_y = row_grain(a.y, a.cols, e);
  k.g_w = row_grain(a.weight, 0, 1);
  if (a.in == InType::BF16)
    return a.codes || a.amax ? pick_norm<true, true>(k, dev, stream)
                             : pick_norm<true, false>(k, dev, stream);
  return a.codes || a.amax ? pick_norm<false, true>(k, dev, stream)
                           : pick_norm<false, false>(k, dev, stream);
}

int64_t add_rmsnorm_backward_workspace(int64_t rows, int64_t cols) {
  // one row of partial sums per CTA; no more CTAs than kNormBackwardParts, nor than rows
  return 4 * cols * std::min<int64_t>(rows, kNormBackwardParts);
}

cudaError_t launch_add_rmsnorm_backward(const NormBackwardArgs& a, const DeviceInfo& dev,
                                        cudaStream_t stream) {
  if (a.cols == 0) return cudaSuccess;
  if (a.rows == 0)
    return a.dweight ? cudaMemsetAsync(a.dweight, 0, 4 * a.cols, stream) : cudaSuccess;
  const int e = a.in == InType::BF16 ? 2 : 4;
  NormBackwardKernelArgs k{};
  k.dy = a.dy;
  k.h = a.h;
  k.dh = a.dh;
  k.w = a.weight;
  k.rstd = a.rstd;
  k.dx = a.dx;
  k.part = a.dweight ? static_cast<float*>(a.workspace) : nullptr;
  k.rows = a.rows;
  k.cols = (int)a.cols;
  k.w_bf16 = a.weight_bf16;
  k.g_dy = row_grain(a.dy, a.cols, e);
  k.g_h = row_grain(a.h, a.cols, e);
  k.g_dh = row_grain(a.dh, a.cols, e);
  k.g_dx = row_grain(a.dx, a.cols, e);
  k.g_w = row_grain(a.weight, 0, 1);
  int parts = 0;
  const int max_parts = (int)std::min<int64_t>(a.rows, kNormBackwardParts);
  cudaError_t err = a.in == InType::BF16
                        ? pick_norm_backward<true>(k, max_parts, dev, stream, &parts)
                        : pick_norm_backward<false>(k, max_parts, dev, stream, &parts);
  if (err != cudaSuccess || a.dweight == nullptr) return err;
  return launch_column_sum(k.part, parts, a.cols, a.dweight, stream);
}

}  // namespace nvfp4
