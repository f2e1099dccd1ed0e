// kernels_layernorm.cu -- dropout, residual addition and layer norm with a quantized output.
//
//   h = residual + drop(x),  m = mean(h),  s = 1 / sqrt(mean((h - m)^2) + eps),
//   y = (h - m) s w + b
//
// The variance is that of the differences, not a difference of moments: each warp takes its
// own mean from registers, sums the squares around it, and the warps' (sum, squares) join
// around the row's mean (Chan, Golub, LeVeque, "Updating formulae and a pairwise algorithm for
// computing sample variances", 1979), so one barrier is enough and a row far from zero loses
// nothing.  The scale of a whole row needs max|y|, which b makes known only after s: a second
// barrier, for those outputs alone.  The rest is norm_rows.cuh's.
#include "norm_rows.cuh"

namespace nvfp4 {
namespace {

// Mean and sum of squared differences of a row whose part is in v (zeros past its end).
template <int TPR, int NCH, bool BARRIER>
__device__ __forceinline__ float2 team_moments(const float (&v)[NCH][kChunk], int cols, int t,
                                               float2* red) {
  const int lane = threadIdx.x & 31, first = t - lane;  // of this warp in its team
  // columns of the warp that starts at thread `from` of the team
  auto count = [&](int from) {
    int n = 0;
#pragma unroll
    for (int c = 0; c < NCH; ++c) n += max(0, min(32 * kChunk, cols - (c * TPR + from) * kChunk));
    return n;
  };
  Pair two = {0.0f, 0.0f};
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int i = 0; i < kChunk; i += 2) two = pair_add(two, {v[c][i], v[c][i + 1]});
  float sum = __fadd_rn(two.x, two.y);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, d));
  const int mine = count(first);
  const float mean = mine > 0 ? __fdiv_rn(sum, (float)mine) : 0.0f;
  two = {0.0f, 0.0f};
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int n = cols - (c * TPR + t) * kChunk;
    if (n >= kChunk) {
#pragma unroll
      for (int i = 0; i < kChunk; i += 2) {
        const Pair d = pair_add({v[c][i], v[c][i + 1]}, {-mean, -mean});
        two = pair_fma(d, d, two);
      }
    } else if (n > 0) {
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        const float d = i < n ? __fsub_rn(v[c][i], mean) : 0.0f;
        two.x = __fmaf_rn(d, d, two.x);
      }
    }
  }
  float sq = __fadd_rn(two.x, two.y);
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) sq = __fadd_rn(sq, __shfl_xor_sync(0xffffffffu, sq, d));
  if constexpr (TPR == 32) {
    if constexpr (BARRIER) __syncthreads();
    return make_float2(mean, sq);
  } else {
    constexpr int kWarps = TPR / 32;
    constexpr int kTree = kWarps <= 2 ? 2 : kWarps <= 4 ? 4 : kWarps <= 8 ? 8 : kWarps <= 16 ? 16 : 32;
    const int warp = threadIdx.x >> 5;
    if (lane == 0) red[warp] = make_float2(sum, sq);
    __syncthreads();
    const int i = lane % kTree;
    const float2 p = i < kWarps ? red[warp - warp % kWarps + i] : make_float2(0.0f, 0.0f);
    const int n = i < kWarps ? count(32 * i) : 0;
    float all = p.x;
#pragma unroll
    for (int d = kTree / 2; d > 0; d >>= 1) all = __fadd_rn(all, __shfl_xor_sync(0xffffffffu, all, d));
    const float m = cols > 0 ? __fdiv_rn(all, (float)cols) : 0.0f;
    const float off = n > 0 ? __fsub_rn(__fdiv_rn(p.x, (float)n), m) : 0.0f;
    float s = __fmaf_rn(__fmul_rn(off, off), (float)n, p.y);
#pragma unroll
    for (int d = kTree / 2; d > 0; d >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, d));
    return make_float2(m, s);
  }
}

// Maximum over a team; red as in team_sum_max.
template <int TPR>
__device__ __forceinline__ float team_max(float m, float* red) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  if constexpr (TPR > 32) {
    constexpr int kWarps = TPR / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) red[warp] = m;
    __syncthreads();
    m = lane < kWarps ? red[warp - warp % kWarps + lane] : 0.0f;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  }
  return m;
}

struct LayerNorm {
  static constexpr bool kMasked = true;
  template <bool BF16, int TPR, int NCH>
  static constexpr int ring_ctas() {
    return 1;
  }

  template <bool BF16, bool NV4, int TPR, int NCH, bool STAGED, bool RING, class Release>
  __device__ __forceinline__ static void row(const NormKernelArgs& a, int64_t row, bool live,
                                             bool has, int t, uint8_t* stage,
                                             float (&v)[NCH][kChunk], float2* red,
                                             const Release& release) {
    // beside red, which the next row's statistics may take while this row's maxima are read
    __shared__ float maxima[TPR < 256 ? 8 : TPR / 32];
    const int64_t base = row * a.cols;
    // past a row's end: the mask's zeros
    if (a.h != nullptr) {
#pragma unroll
      for (int c = 0; c < NCH; ++c)
        store_row<BF16, TPR, NCH, STAGED>(a, a.h, a.g_h, base, has, t, stage, c, v[c]);
    }
    const float2 r = team_moments<TPR, NCH, RING>(v, a.cols, t, red);
    if (!release()) return;
    const float var = a.cols > 0 ? __fdiv_rn(r.y, (float)a.cols) : 0.0f;
    const float s = __frsqrt_rn(__fadd_rn(var, a.eps));
    if (live && t == 0) {
      if (a.mean != nullptr) a.mean[row] = r.x;
      if (a.rstd != nullptr) a.rstd[row] = s;
    }
    const bool quantized = NV4 || a.q8 != nullptr;
    float bmax[NCH], mx = 0.0f;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int col = (c * TPR + t) * kChunk, n = chunk_len(col, a.cols);
      float w[kChunk], b[kChunk];
      load_vector16(a.w, a.w_bf16, col, n, a.g_w, w);
      if (a.b != nullptr) {
        load_vector16(a.b, a.w_bf16, col, n, a.g_b, b);
      } else {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) b[i] = 0.0f;
      }
      bmax[c] = 0.0f;
#pragma unroll
      for (int i = 0; i < kChunk; i += 2) {  // w and b are zero past the row's end
        const Pair n2 = pair_mul(pair_add({v[c][i], v[c][i + 1]}, {-r.x, -r.x}), {s, s});
        const Pair y = pair_fma(n2, {w[i], w[i + 1]}, {b[i], b[i + 1]});
        v[c][i] = y.x;
        v[c][i + 1] = y.y;
        if (quantized) bmax[c] = fmaxf(fmaxf(bmax[c], fabsf(y.x)), fabsf(y.y));
      }
      mx = fmaxf(mx, bmax[c]);
    }
    if (NV4 ? a.amax_in == nullptr : quantized && !a.q8_blocks) mx = team_max<TPR>(mx, maxima);
    emit_row<BF16, NV4, TPR, NCH, STAGED>(a, row, live, t, stage, v, mx,
                                          [&](int c) { return bmax[c]; });
  }
};

}  // namespace

cudaError_t launch_add_layernorm(const NormArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  return launch_norm<LayerNorm>(a, dev, stream);
}

}  // namespace nvfp4
