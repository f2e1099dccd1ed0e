// kernels_norm.cu -- residual addition and root-mean-square norm with a quantized output.
//
//   h = x + residual,  s = 1 / sqrt(mean(h^2) + eps),  y = h * w * s
//
// The statistic and the row's amax come out of one reduction: amax(y) = s max|h w| exactly,
// because rounding after the product with the positive s is monotonic; the scale of the whole
// row is therefore known one barrier after its last load.  The rest is norm_rows.cuh's.
//
// Measured (E4M3 output, residual): 16384 x 8192 BF16 143 us, 6.6 TB/s, 0.98 of a copy (182
// us without the ring), NVFP4 rows 144 us; 4000 x 5000 FP32 in 128-column blocks 47 us, 5.6
// TB/s (barriers and shared-memory rotations are in sight there: issue slots are 54 % used);
// one row of 8192 3.0 us, which is a launch and one pass of latencies.
#include "norm_rows.cuh"

namespace nvfp4 {
namespace {

// The maximum of |h w| s over values of |h w| up to m, NaN skipped: 0 where the product is one
// (m infinite and s = 0, a row whose only value other than 0 is NaN; m = 0 and s infinite).
__device__ __forceinline__ float amax_times(float m, float s) {
  return fmaxf(__fmul_rn(m, s), 0.0f);
}

struct RmsNorm {
  static constexpr bool kMasked = false;
  using Sums = float2;
  template <bool BF16, int TPR, int NCH>
  static constexpr int ring_ctas() {
    return 1;
  }
  // 16384 x 8192 BF16 with a residual and a scale per row: two CTAs of three stages an SM 145 us, three
  // of two 154
  template <int NCH>
  static constexpr int third_cta() {
    return NCH == 2 ? 3 : 2;
  }

  template <int TPR, int NCH>
  struct Team;
};

template <int TPR, int NCH>
struct RmsNorm::Team {
  __device__ __forceinline__ Team(const NormKernelArgs&, int) {}
  // has: the row's values arrived (they have not where a bounded wait gave up)
  template <bool BF16, bool NV4, bool STAGED, bool RING, class Release>
  __device__ __forceinline__ void row(const NormKernelArgs& a, int64_t row, bool live, bool has,
                                      int t, uint8_t* stage, float (&v)[NCH][kChunk], float2* red,
                                      const Release& release) const {
    const int64_t base = row * a.cols;
    // h out, then h w with the sum of h^2 and the maxima of |h w|
    float bmax[NCH], ss = 0.0f, mx = 0.0f;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int col = (c * TPR + t) * kChunk;
      if (a.h != nullptr)
        store_row<BF16, TPR, NCH, STAGED>(a, a.h, a.g_h, base, has, t, stage, c, v[c]);
      float w[kChunk];
      load_vector16(a.w, a.w_bf16, col, has ? chunk_len(col, a.cols) : 0, a.g_w, w);
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
    const float2 r = team_sum_max<TPR, RING>(ss, mx, red);
    if (!release()) return;
    const float mean = a.cols > 0 ? __fdiv_rn(r.x, (float)a.cols) : 0.0f;
    const float s = __frsqrt_rn(__fadd_rn(mean, a.eps));
    if (live && t == 0 && a.rstd != nullptr) a.rstd[row] = s;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int i = 0; i < kChunk; ++i) v[c][i] = __fmul_rn(v[c][i], s);
    emit_row<BF16, NV4, TPR, NCH, STAGED>(a, row, live, t, stage, v, amax_times(r.y, s),
                                          [&](int c) { return amax_times(bmax[c], s); });
  }
};

}  // namespace

cudaError_t launch_add_rmsnorm(const NormArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  return launch_norm<RmsNorm>(a, dev, stream);
}

}  // namespace nvfp4
