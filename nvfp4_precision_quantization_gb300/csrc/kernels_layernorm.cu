// kernels_layernorm.cu -- dropout, residual addition and layer norm with a quantized output.
//
//   h = residual + drop(x),  m = mean(h),  s = 1 / sqrt(mean((h - m)^2) + eps),
//   y = (h - m) s w + b
//
// The variance is that of the differences, not a difference of moments.  Each warp takes its own mean m_w
// from registers, then the sums e_w of its n_w differences to it and Q_w of their squares.  With off =
// m_w - m, for any m near the row's values, the row's are
//   sum (h - m) = e_w + n_w off,   sum (h - m)^2 = Q_w + 2 off e_w + n_w off^2
// (Chan, Golub, LeVeque, "Updating formulae and a pairwise algorithm for computing sample
// variances", 1979, where e_w is 0; m_w is rounded here, and without e_w rows of 65536 +- 1 lost 2e-4
// of their variance), and the first moves m to the row's mean and takes its part off the second.  m is
// the mean of the team's first warp where that is beyond one of its standard deviations, and 0 in rows
// that lie around 0, whose sum of values is the better mean.  Either way it is within 2 / sqrt(f) of the
// row's standard deviations of its mean, f >= 1/32 being the first warp's share (mostly within a
// few hundredths, or one): so much is what is taken off, at most, beside what is left.  One barrier is
// enough, and a row far from zero loses nothing but its own rounding.  The scale of a whole row needs
// max|y|, which b makes known only after s: a second barrier, for those outputs alone.  The rest is
// norm_rows.cuh's.
//
// Measured (residual, bias): 4000 x 5000 FP32 54 us, 5.9 TB/s; 16384 x 8192 BF16 with E4M3 codes or
// NVFP4 rows 186 us, 5.1 and 4.7 TB/s, and 242 us with dropout.  BF16 rows stop at 31 instructions an
// element (25 with y alone, 170 us) and 12 more for the mask, in 55 to 60 % of the issue slots: the
// rest is latency that 24 warps an SM with two barriers a row leave open.  The differences' sums and
// their join are 1.5 of the instructions and 4 % of those times.  One row of 8192 4 us.
#include "norm_rows.cuh"

namespace nvfp4 {
namespace {

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
  // of values; of squared differences to their mean and of differences; the mean
  using Sums = float4;
  // 24 warps an SM: with the 16 that the compiler's registers leave, a row's barriers lie open
  // (4000 x 5000 FP32 74 us, 53 so); 16 for two FP32 chunks a thread, which spill (16000 x 8192 FP32
  // 460 us with 24, 416 with 16)
  template <bool BF16, int TPR, int NCH>
  static constexpr int ring_ctas() {
    constexpr int n = (!BF16 && NCH == 2 ? 512 : 768) / (TPR < 256 ? 256 : TPR);
    return n > 0 ? n : 1;
  }
  template <int NCH>
  static constexpr int third_cta() {
    return 2;
  }
  template <int TPR, int NCH>
  struct Team;
};

template <int TPR, int NCH>
struct LayerNorm::Team {
  static constexpr int kWarps = TPR / 32;
  static constexpr int kTree = kWarps <= 1 ? 1 : kWarps <= 2 ? 2 : kWarps <= 4 ? 4 : kWarps <= 8 ? 8 : kWarps <= 16 ? 16 : 32;
  float inv_warp;   // 1 / the columns of this thread's warp (0 where it has none)
  float n, n_first; // those of the team's warp `lane`, whose sums this lane joins, and of its first one
  float inv_cols;

  // columns of the team's warp w
  __device__ __forceinline__ static int count(int cols, int w) {
    int n = 0;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
      n += max(0, min(32 * kChunk, cols - (c * TPR + 32 * w) * kChunk));
    return n;
  }
  __device__ __forceinline__ static float inverse(int n) {
    return n > 0 ? __frcp_rn((float)n) : 0.0f;
  }
  __device__ __forceinline__ Team(const NormKernelArgs& a, int t) {
    const int w = (threadIdx.x & 31) % kTree, theirs = w < kWarps ? count(a.cols, w) : 0;
    inv_warp = inverse(count(a.cols, t / 32));
    n = (float)theirs;
    n_first = (float)count(a.cols, 0);
    inv_cols = inverse(a.cols);
  }

  // A sum over the lanes of two values at once, N lanes each: lane l gets that of a where l & (N / 2)
  // is 0, and that of b elsewhere.
  template <int N>
  __device__ __forceinline__ static float sum_of_two(float a, float b, int lane) {
    const bool upper = lane & (N / 2);
    const float keep = upper ? b : a, give = upper ? a : b;
    float s = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, give, N / 2));
#pragma unroll
    for (int d = N / 4; d > 0; d >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, d));
    return s;
  }
  __device__ __forceinline__ static bool finite(float x) {
    return fabsf(x) < __int_as_float(0x7f800000);
  }
  // The sum of squared differences to the mean, from sums of differences to some m and of their squares
  // (not below 0 but for its rounding; an infinity or a NaN stays).
  __device__ __forceinline__ float around_mean(float rest, float sq) const {
    float s = __fmaf_rn(-rest, __fmul_rn(rest, inv_cols), sq);
    asm("max.NaN.f32 %0, %0, 0f00000000;" : "+f"(s));
    return s;
  }

  // Mean and sum of squared differences of a row whose part is in v (zeros past its end).
  template <bool BARRIER>
  __device__ __forceinline__ float2 moments(const float (&v)[NCH][kChunk], int cols, int t,
                                            Sums* red) const {
    const int lane = threadIdx.x & 31;
    Pair two = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int i = 0; i < kChunk; i += 2) two = pair_add(two, {v[c][i], v[c][i + 1]});
    float sum = __fadd_rn(two.x, two.y);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, d));
    const float mean = __fmul_rn(sum, inv_warp);
    Pair rest = {0.0f, 0.0f};
    two = {0.0f, 0.0f};
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int left = cols - (c * TPR + t) * kChunk;
      if (left >= kChunk) {
#pragma unroll
        for (int i = 0; i < kChunk; i += 2) {
          const Pair d = pair_add({v[c][i], v[c][i + 1]}, {-mean, -mean});
          rest = pair_add(rest, d);
          two = pair_fma(d, d, two);
        }
      } else if (left > 0) {
#pragma unroll
        for (int i = 0; i < kChunk; ++i) {
          const float d = i < left ? __fsub_rn(v[c][i], mean) : 0.0f;
          rest.x = __fadd_rn(rest.x, d);
          two.x = __fmaf_rn(d, d, two.x);
        }
      }
    }
    // squares in the lower lanes, differences in the upper ones
    const float both =
        sum_of_two<32>(__fadd_rn(two.x, two.y), __fadd_rn(rest.x, rest.y), lane);
    if constexpr (TPR == 32) {
      if constexpr (BARRIER) __syncthreads();
      const float other = __shfl_xor_sync(0xffffffffu, both, 16);
      const float sq = lane < 16 ? both : other, rest = lane < 16 ? other : both;
      const bool far = __fmul_rn(mean, mean) > __fmul_rn(sq, inv_cols);  // not where it is infinite
      return make_float2(far ? __fmaf_rn(rest, inv_cols, mean) : mean, around_mean(rest, sq));
    } else {
      const int warp = threadIdx.x >> 5, first = warp - warp % kWarps;
      if (lane == 0) {
        red[warp].x = sum;
        red[warp].y = both;
        red[warp].w = mean;
      } else if (lane == 16) {
        red[warp].z = both;
      }
      __syncthreads();
      const float4 own = red[first];
      // (a NaN is not beyond)
      const float m = __fmul_rn(__fmul_rn(own.w, own.w), n_first) > own.y ? own.w : 0.0f;
      // this lane's warp's differences to m
      const int i = lane % kTree;
      const float4 p = i < kWarps ? red[first + i] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      const float off = n > 0.0f ? __fsub_rn(p.w, m) : 0.0f;  // (0: a warp without columns)
      const float sq = __fmaf_rn(__fmul_rn(off, off), n, __fmaf_rn(__fadd_rn(off, off), p.z, p.y));
      // (a sum that is no number has no differences, and stands for them)
      const float rest = m != 0.0f && finite(p.x) ? __fmaf_rn(off, n, p.z) : p.x;
      const float joined = sum_of_two<kTree>(sq, rest, lane);
      const float other = __shfl_xor_sync(0xffffffffu, joined, kTree / 2);
      const bool upper = lane & (kTree / 2);
      const float all = upper ? joined : other;
      return make_float2(__fmaf_rn(all, inv_cols, m), around_mean(all, upper ? other : joined));
    }
  }

  // v = (v - m) s w + b of 16 columns (w and b are zero past the row's end); their largest |y|.
  template <bool WEIGHT_BF16>
  __device__ __forceinline__ static float affine(const NormKernelArgs& a, int col, float m,
                                                 float s, float (&v)[kChunk]) {
    const int n = chunk_len(col, a.cols);
    Chunk<WEIGHT_BF16> w, b;
    w.load(a.w, col, n, a.g_w);
    b.load(a.b, col, a.b != nullptr ? n : 0, a.g_b);
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < kChunk; i += 2) {
      const Pair d = pair_mul(pair_add({v[i], v[i + 1]}, {-m, -m}), {s, s});
      const Pair y = pair_fma(d, {w.get(i), w.get(i + 1)}, {b.get(i), b.get(i + 1)});
      v[i] = y.x;
      v[i + 1] = y.y;
      asm("max.abs.f32 %0, %0, %1, %2;" : "+f"(top) : "f"(y.x), "f"(y.y));  // NaN skipped
    }
    return top;
  }

  template <bool BF16, bool NV4, bool STAGED, bool RING, class Release>
  __device__ __forceinline__ void row(const NormKernelArgs& a, int64_t row, bool live, bool has,
                                      int t, uint8_t* stage, float (&v)[NCH][kChunk], Sums* red,
                                      const Release& release) const {
    // beside red, which the next row's statistics may take while this row's maxima are read
    __shared__ float maxima[TPR < 256 ? 8 : TPR / 32];
    const int64_t base = row * a.cols;
    if (a.h != nullptr) {
#pragma unroll
      for (int c = 0; c < NCH; ++c)
        store_row<BF16, TPR, NCH, STAGED>(a, a.h, a.g_h, base, has, t, stage, c, v[c]);
    }
    const float2 r = moments<RING>(v, a.cols, t, red);
    if (!release()) return;
    const float s = __frsqrt_rn(__fmaf_rn(r.y, inv_cols, a.eps));
    if (live && t == 0) {
      if (a.mean != nullptr) a.mean[row] = r.x;
      if (a.rstd != nullptr) a.rstd[row] = s;
    }
    const bool quantized = NV4 || a.q8 != nullptr;
    float bmax[NCH], mx = 0.0f;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int col = (c * TPR + t) * kChunk;
      bmax[c] = a.w_bf16 ? affine<true>(a, col, r.x, s, v[c]) : affine<false>(a, col, r.x, s, v[c]);
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
