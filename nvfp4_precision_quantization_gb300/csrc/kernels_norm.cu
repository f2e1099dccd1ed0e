// kernels_norm.cu -- residual addition and root-mean-square norm with a quantized output.
//
//   h = x + residual,  s = 1 / sqrt(mean(h^2) + eps),  y = h * w * s
//
// Bound by memory: every tensor is read or written once.  A row's team of
// threads holds the row in registers (16 consecutive elements per thread and step), so
// neither the statistic nor the row's amax needs a second read.  Both come out
// of one reduction: amax(y) = s max|h w| exactly, because rounding after the product
// with the positive s is monotonic; the scale of the whole row is therefore known one
// barrier after its last load.
//
// Measured (E4M3 output, residual): 16384 x 8192 BF16 147 us, 6.4 TB/s, 0.96 of a copy (182
// us without the ring), NVFP4 rows 153 us; 4000 x 5000 FP32 in 128-column blocks 49 us, 5.3
// TB/s (barriers and shared-memory rotations are in sight there: issue slots are 54 % used);
// one row of 8192 3.0 us, which is a launch and one pass of latencies.
#include "row_ring.cuh"

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
  int g_x, g_res, g_w, g_h, g_y, g_q8, g_codes;  // row grains (row_io.cuh)
  int g_min;  // the least of those of x, res, h, y (and of codes below 4)
  bool bases_aligned;  // x and res start on 16 bytes
  int* status;
};

constexpr float kE4m3Max = 448.0f;

// The maximum of |h w| s over values of |h w| up to m, NaN skipped: 0 where the product is one
// (m infinite and s = 0, a row whose only value other than 0 is NaN; m = 0 and s infinite).
__device__ __forceinline__ float amax_times(float m, float s) {
  return fmaxf(__fmul_rn(m, s), 0.0f);
}

// The scale of an E4M3 output whose largest magnitude is a.
__device__ __forceinline__ float fp8_scale(float a) {
  return a == 0.0f ? 1.0f : fmaxf(__fdiv_rn(a, kE4m3Max), 0x1p-126f);
}
// Quotients by such a scale: the codes are those of y / scale, whatever the scale's rounding
// and its lower bound make of it (codes of y * (448 / a) decoded to up to four times y for a
// below 448 * 2^-126, and lay up to three roundings from the quotient otherwise).
// q = y r with r = 1 / scale, and one Newton step on the residual y - q scale, which an FMA
// gives exactly (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990): 16 divisions would cost five times the instructions.
struct Fp8Divisor {
  float r, minus;  // 1 / scale, and -scale (0 for an infinite one: the step adds nothing to 0)
};
__device__ __forceinline__ Fp8Divisor fp8_divisor(float scale) {
  return {__frcp_rn(scale), isinf(scale) ? 0.0f : -scale};
}
__device__ __forceinline__ Pair fp8_quotient(Pair y, const Fp8Divisor& d) {
  const Pair q = pair_mul(y, {d.r, d.r});
  const Pair rest = pair_fma(q, {d.minus, d.minus}, y);
  return pair_fma(rest, {d.r, d.r}, q);
}

// What a thread does with its part of a row once h is in v: h out, then h w with the sum
// of h^2 and the maxima of |h w| (bmax per chunk).
template <bool BF16, int TPR, int NCH, bool STAGED>
__device__ __forceinline__ void norm_gather(const NormKernelArgs& a, int64_t base, bool live, int t,
                                            uint8_t* stage, float (&v)[NCH][kChunk],
                                            float (&bmax)[NCH], float& ss, float& mx) {
  const int lane = threadIdx.x & 31;
  ss = mx = 0.0f;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int col = (c * TPR + t) * kChunk;
    const int n = live ? chunk_len(col, a.cols) : 0;
    if (a.h != nullptr) {
      Chunk<BF16> ch;
      ch.set(v[c]);
      ch.store_warp<STAGED>(a.h, base + col, n,
                            live ? warp_run(col - kChunk * lane, a.cols) : 0, a.g_h, stage,
                            lane);
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
}

// The outputs of a row whose team found sum(h^2) = r.x and max|h w| = r.y.
template <bool BF16, bool NV4, int TPR, int NCH, bool STAGED>
__device__ __forceinline__ void norm_emit(const NormKernelArgs& a, int64_t row, bool live, int t,
                                          uint8_t* stage, float (&v)[NCH][kChunk],
                                          const float (&bmax)[NCH], float2 r) {
  const int lane = threadIdx.x & 31;
  const int64_t base = row * a.cols;
  const float mean = a.cols > 0 ? __fdiv_rn(r.x, (float)a.cols) : 0.0f;
  const float s = __frsqrt_rn(__fadd_rn(mean, a.eps));
  const float top = amax_times(r.y, s);  // amax of the row's y
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
      cy.store_warp<STAGED>(a.y, base + col, live ? chunk_len(col, a.cols) : 0,
                            live ? warp_run(col - kChunk * lane, a.cols) : 0, a.g_y, stage,
                            lane);
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
      const float b = amax_times(bmax[c], s);
      uint32_t cw[2] = {0, 0};
      uint32_t s8 = 0;
      if (n == 0) {  // nothing of the row
      } else if (a.four_over_six)
        s8 = quantize16<true>(v[c], b, S, line, a.F_inv, a.negz, cw[0], cw[1]);
      else
        s8 = quantize16<false>(v[c], b, S, line, a.F_inv, a.negz, cw[0], cw[1]);
      uint8_t* codes = a.codes + row * cpitch + col / 2;
      if (!STAGED || a.g_codes >= 4) {
        if (n > 0) store_bytes(codes, cw, (n + 1) / 2);
      } else {
        staged_store<2, 8, 1, 2>(reinterpret_cast<char*>(codes) - 8 * lane,
                           live ? ((int)warp_run(col - kChunk * lane, a.cols) + 1) / 2 : 0,
                           a.g_codes, stage, lane, cw);
      }
      if (n > 0) a.scales[row * spitch + col / 16] = (uint8_t)s8;
    }
  } else if (a.q8 != nullptr) {
    const float s_row = fp8_scale(top);
    if (live && t == 0 && !a.q8_blocks) a.q8_scale[row] = s_row;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int col = (c * TPR + t) * kChunk;
      const int n = live ? chunk_len(col, a.cols) : 0;
      float scale = s_row;
      if (a.q8_blocks) {  // 128 columns are eight neighbouring lanes
        float b = bmax[c];
#pragma unroll
        for (int d = 4; d > 0; d >>= 1) b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, d));
        b = amax_times(b, s);
        scale = fp8_scale(b);
        if (n > 0 && (t & 7) == 0)
          a.q8_scale[row * ((a.cols + 127) / 128) + col / 128] = scale;
      }
      const Fp8Divisor d = fp8_divisor(scale);
      uint32_t cw[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const Pair a01 = fp8_quotient({v[c][4 * i], v[c][4 * i + 1]}, d);
        const Pair a23 = fp8_quotient({v[c][4 * i + 2], v[c][4 * i + 3]}, d);
        uint16_t lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(a01.y), "f"(a01.x));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(a23.y), "f"(a23.x));
        cw[i] = (uint32_t)lo | ((uint32_t)hi << 16);
      }
      if (!STAGED || a.g_q8 >= 4) {
        if (n > 0) store_bytes(a.q8 + base + col, cw, n);
      } else {
        shifted_store(reinterpret_cast<char*>(a.q8) + base + col - kChunk * lane,
                      live ? (int)warp_run(col - kChunk * lane, a.cols) : 0, lane, cw);
      }
    }
  }
}

// Rows straight from memory into registers: few rows (each CTA has one or two, so there
// is nothing to run ahead of), and (STAGED) unaligned ones that the ring does not take: rows of
// more than 16384 columns, BF16 rows of one warp's team, tensors that do not start on 16 bytes.
template <bool BF16, bool NV4, int TPR, int NCH, bool STAGED>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR) k_add_rmsnorm(const NormKernelArgs a) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  constexpr int kTeams = kThreads / TPR;
  __shared__ float2 red[2][kThreads / 32];
  __shared__ __align__(16) uint8_t stages[STAGED ? kThreads / 32 : 1][kStageBytes];
  const int t = threadIdx.x % TPR, team = threadIdx.x / TPR, lane = threadIdx.x & 31;
  uint8_t* stage = stages[STAGED ? threadIdx.x >> 5 : 0];
  int buf = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * kTeams; row0 < a.rows;
       row0 += (int64_t)gridDim.x * kTeams, buf ^= 1) {
    const int64_t row = row0 + team;
    const bool live = row < a.rows;
    const int64_t base = row * a.cols;
    float v[NCH][kChunk], bmax[NCH], ss, mx;
    ChunkLoad<BF16, STAGED> lx[NCH], lr[NCH];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int col = (c * TPR + t) * kChunk;
      const int n = live ? chunk_len(col, a.cols) : 0;
      const int64_t run = live ? warp_run(col - kChunk * lane, a.cols) : 0;
      lx[c].issue(a.x, base + col, n, run, a.g_x, lane);
      if (a.res != nullptr) lr[c].issue(a.res, base + col, n, run, a.g_res, lane);
    }
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const Chunk<BF16>& cx = lx[c].settle(a.g_x, stage, lane);
#pragma unroll
      for (int i = 0; i < kChunk; ++i) v[c][i] = cx.get(i);
      if (a.res != nullptr) {
        const Chunk<BF16>& cr = lr[c].settle(a.g_res, stage, lane);
#pragma unroll
        for (int i = 0; i < kChunk; ++i) v[c][i] = __fadd_rn(v[c][i], cr.get(i));
      }
    }
    norm_gather<BF16, TPR, NCH, STAGED>(a, base, live, t, stage, v, bmax, ss, mx);
    const float2 r = team_sum_max<TPR>(ss, mx, red[buf]);
    norm_emit<BF16, NV4, TPR, NCH, STAGED>(a, row, live, t, stage, v, bmax, r);
  }
}

// CTAs per SM that the registers of the kernel for unaligned rows have to allow: left to
// itself the compiler takes up to 168 per thread, and the row's latencies lie open (4000 x 5001
// BF16 76 us with 168, 58 with 80; FP32 86 and 71).
constexpr int ring_any_ctas(bool bf16, int threads) {
  const int n = (bf16 ? 1024 : 768) / threads;
  return n > 0 ? n : 1;
}

// ANY: rows that are not 16-byte aligned (RowRing).
template <bool BF16, bool NV4, int TPR, int NCH, bool ANY>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR,
                                  ANY ? ring_any_ctas(BF16, TPR < 256 ? 256 : TPR) : 1)
    k_add_rmsnorm_ring(const NormKernelArgs a, const RingArgs g) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  constexpr int kTeams = kThreads / TPR;
  constexpr int kElem = BF16 ? 2 : 4;
  extern __shared__ __align__(128) uint8_t ring_smem[];
  __shared__ float2 red[2][kThreads / 32];
  __shared__ __align__(8) uint64_t full[kRingStages];
  __shared__ int err;
  __shared__ __align__(16) uint8_t stages[ANY ? kThreads / 32 : 1][kStageBytes];
  const int t = threadIdx.x % TPR, team = threadIdx.x / TPR, lane = threadIdx.x & 31;
  uint8_t* out_stage = ANY ? stages[ANY ? threadIdx.x >> 5 : 0] : nullptr;
  const int64_t step = (int64_t)gridDim.x * kTeams;
  const RowRing<2, ANY> ring{full, &err, ring_smem, {a.x, a.res}, a.rows,
                             (int64_t)a.cols * kElem, kTeams, g};
  ring.start(step);
  int it = 0, s = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * kTeams; row0 < a.rows; row0 += step, ++it) {
    const int64_t row = row0 + team;
    const bool live = row < a.rows;
    const int64_t base = row * a.cols;
    const uint8_t* st = ring.stage(s) + ring.shift(row0) + team * a.cols * kElem;
    const bool ok = ring.wait(s, it);
    ring.finish(s, row0);
    float v[NCH][kChunk], bmax[NCH], ss, mx;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int col = (c * TPR + t) * kChunk;
      const int n = live && ok ? chunk_len(col, a.cols) : 0;
      Chunk<BF16> cx;
      if constexpr (ANY) {
        cx.load_shared_any(st + min(col, a.cols) * kElem, lane);
        cx.cut(n);
      } else {
        cx.load_shared(st + col * kElem, n, lane);
      }
#pragma unroll
      for (int i = 0; i < kChunk; ++i) v[c][i] = cx.get(i);
      if (a.res != nullptr) {
        Chunk<BF16> cr;
        if constexpr (ANY) {
          cr.load_shared_any(st + g.tensor_bytes + min(col, a.cols) * kElem, lane);
          cr.cut(n);
        } else {
          cr.load_shared(st + g.tensor_bytes + col * kElem, n, lane);
        }
#pragma unroll
        for (int i = 0; i < kChunk; ++i) v[c][i] = __fadd_rn(v[c][i], cr.get(i));
      }
    }
    norm_gather<BF16, TPR, NCH, ANY>(a, base, live && ok, t, out_stage, v, bmax, ss, mx);
    const float2 r = team_sum_max<TPR, true>(ss, mx, red[it & 1]);
    if (*(volatile int*)&err) {
      ring.give_up(it, row0, step, a.status);
      return;
    }
    if (threadIdx.x == 0 && row0 + g.stages * step < a.rows)
      ring.fetch(s, row0 + g.stages * step);
    norm_emit<BF16, NV4, TPR, NCH, ANY>(a, row, live, t, out_stage, v, bmax, r);
    if (++s == g.stages) s = 0;
  }
}

// The direct kernel.
template <bool BF16, bool NV4, int TPR, int NCH, bool STAGED>
cudaError_t run_norm_direct(const NormKernelArgs& k, int64_t groups, const DeviceInfo& dev,
                            cudaStream_t stream) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  const auto kernel = k_add_rmsnorm<BF16, NV4, TPR, NCH, STAGED>;
  static const int resident = resident_ctas(kernel, kThreads);
  const int64_t grid = std::min<int64_t>(groups, (int64_t)resident * dev.num_sms);
  kernel<<<(unsigned)grid, kThreads, 0, stream>>>(k);
  return cudaGetLastError();
}

// The ring kernel, where at least two stages fit and every CTA has several groups (done).
template <bool BF16, bool NV4, int TPR, int NCH, bool ANY>
cudaError_t run_norm_ring(const NormKernelArgs& k, int64_t groups, const DeviceInfo& dev,
                          cudaStream_t stream, bool* done) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  auto ring = k_add_rmsnorm_ring<BF16, NV4, TPR, NCH, ANY>;
  static const RingKernel limits = ring_kernel(ring, kThreads);
  const RingPlan p = plan_ring(limits, k.res ? 2 : 1,
                               (int64_t)(kThreads / TPR) * k.cols * (BF16 ? 2 : 4), ANY);
  const int64_t fill = (int64_t)p.ctas * dev.num_sms;
  if (p.ctas == 0 || groups <= 2 * fill) return cudaSuccess;
  *done = true;
  const cudaError_t e = allow_ring(ring, limits);
  if (e != cudaSuccess) return e;
  ring<<<(unsigned)fill, kThreads, p.g.stages * p.g.stage_bytes, stream>>>(k, p.g);
  return cudaGetLastError();
}

// ROWS: which rows pick_norm sends here (the kernels of the others are not made): aligned ones,
// few or many, or many alone, or those that are not aligned.
enum NormRows { kAnyRows, kFewAlignedOrUnaligned, kManyAligned, kUnaligned };

template <bool BF16, bool NV4, int TPR, int NCH, NormRows ROWS>
cudaError_t run_norm(const NormKernelArgs& k, const DeviceInfo& dev, cudaStream_t stream) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  constexpr int kTeams = kThreads / TPR;
  const int64_t groups = (k.rows + kTeams - 1) / kTeams;
  bool done = false;
  cudaError_t e = cudaSuccess;
  if constexpr (ROWS != kUnaligned) {
    if (k.g_min >= 16) {
      // few rows: one or two for each CTA, so never through the ring
      if constexpr (ROWS != kFewAlignedOrUnaligned)
        e = run_norm_ring<BF16, NV4, TPR, NCH, false>(k, groups, dev, stream, &done);
      if (done || e != cudaSuccess) return e;
      return run_norm_direct<BF16, NV4, TPR, NCH, false>(k, groups, dev, stream);
    }
  }
  if constexpr (ROWS != kManyAligned) {
    // Rows that are not aligned: one step per thread (two stages of longer rows seldom fit).
    // Through the ring and loaded directly, BF16 with FP8 codes: 4000 x 5001 59 and 80 us,
    // 16384 x 1001 42 and 88; FP32: 4000 x 5001 69 and 103, 16384 x 511 30 and 41.  BF16
    // rows of one warp's team do not gain: 16384 x 500 25.4 and 22.6, 16384 x 511 26.7 and 25.8.
    if constexpr (NCH == 1 && (TPR > 32 || !BF16)) {
      if (k.bases_aligned)
        e = run_norm_ring<BF16, NV4, TPR, NCH, true>(k, groups, dev, stream, &done);
      if (done || e != cudaSuccess) return e;
    }
    return run_norm_direct<BF16, NV4, TPR, NCH, true>(k, groups, dev, stream);
  }
  return cudaErrorInvalidValue;  // not reached: pick_norm sends no other rows here
}

template <bool BF16, bool NV4>
cudaError_t pick_norm(const NormKernelArgs& k, const DeviceInfo& dev, cudaStream_t stream) {
  // one step of 16 elements per thread while the rows do not fill the GPU, two beyond; one
  // for staged rows, whose loads in flight take twice the registers
  const bool few = k.rows <= 2LL * dev.num_sms || k.g_min < 16;
  const int c = k.cols;
  if (c <= 512) return run_norm<BF16, NV4, 32, 1, kAnyRows>(k, dev, stream);
  // teams of two warps where those of four would be half idle (16384 x 1001 unaligned: 41 us,
  // and 76 by four)
  if (c <= 1024 && k.g_min < 16) return run_norm<BF16, NV4, 64, 1, kUnaligned>(k, dev, stream);
  if (c <= 1024 && !few) return run_norm<BF16, NV4, 32, 2, kManyAligned>(k, dev, stream);
  if (c <= 2048) return run_norm<BF16, NV4, 128, 1, kAnyRows>(k, dev, stream);
  if (c <= 4096) return run_norm<BF16, NV4, 256, 1, kAnyRows>(k, dev, stream);
  if (c <= 6144) return run_norm<BF16, NV4, 384, 1, kAnyRows>(k, dev, stream);
  if (c <= 8192 && !few) return run_norm<BF16, NV4, 256, 2, kManyAligned>(k, dev, stream);
  if (c <= 8192) return run_norm<BF16, NV4, 512, 1, kFewAlignedOrUnaligned>(k, dev, stream);
  if (c <= 16384 && !few) return run_norm<BF16, NV4, 512, 2, kManyAligned>(k, dev, stream);
  if (c <= 16384) return run_norm<BF16, NV4, 1024, 1, kFewAlignedOrUnaligned>(k, dev, stream);
  return run_norm<BF16, NV4, 1024, 2, kAnyRows>(k, dev, stream);
}

}  // namespace

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
  k.g_x = row_grain(a.x, a.cols * e);
  k.g_res = row_grain(a.residual, a.cols * e);
  k.g_h = row_grain(a.h, a.cols * e);
  k.g_y = row_grain(a.y, a.cols * e);
  k.g_w = row_grain(a.weight, 0);
  k.g_q8 = row_grain(a.q8, a.cols);
  k.g_codes = row_grain(a.codes, (a.cols + 1) / 2);
  k.g_min = k.g_x;  // tensors that are not given do not count
  if (a.residual) k.g_min = std::min(k.g_min, k.g_res);
  if (a.h) k.g_min = std::min(k.g_min, k.g_h);
  if (a.y) k.g_min = std::min(k.g_min, k.g_y);
  // (codes are stored in words where they are so aligned)
  if (a.q8 && k.g_q8 < 4) k.g_min = std::min(k.g_min, k.g_q8);
  if (a.codes && k.g_codes < 4) k.g_min = std::min(k.g_min, k.g_codes);
  k.bases_aligned =
      (reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.residual)) % 16 == 0;
  k.status = dev.status;
  if (a.in == InType::BF16)
    return a.codes || a.amax ? pick_norm<true, true>(k, dev, stream)
                             : pick_norm<true, false>(k, dev, stream);
  return a.codes || a.amax ? pick_norm<false, true>(k, dev, stream)
                           : pick_norm<false, false>(k, dev, stream);
}

}  // namespace nvfp4
