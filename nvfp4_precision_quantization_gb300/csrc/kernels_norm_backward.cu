// kernels_norm_backward.cu -- gradients of the residual addition and root-mean-square norm.
//
//   dx = s (g - n mean(g n)) + dh,  dw = sum_rows dy n,   n = h s,  g = dy w
//
// Bound by memory: every tensor is read or written once.  A row's team of threads holds dy,
// h and dh in registers across the one reduction that the row needs, and each thread the
// weight's gradient of its columns across all rows of its CTA.
//
// Measured: 16384 x 8192 BF16 with dh 176 us, 6.1 TB/s, 0.91 of a copy (266 us without the
// ring); 4000 x 5000 FP32 51 us, 4.7 TB/s (313 of a team's 384 threads have columns, and the
// dw sums are joined by a second launch of 3 us).
#include "row_ring.cuh"

namespace nvfp4 {
namespace {

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
  int g_dy, g_h, g_dh, g_w, g_dx, g_part;
  int g_min;  // the least of those of dy, h, dh and dx
  bool bases_aligned;  // dy, h and dh start on 16 bytes
  int* status;
};

// dw of the columns of a thread and the row's sum of g n, from dy and h of a row.
template <bool BF16, int TPR, int NCH>
__device__ __forceinline__ float backward_gather(const NormBackwardKernelArgs& a, int t, float s,
                                                 const Chunk<BF16> (&cy)[NCH],
                                                 const Chunk<BF16> (&ch)[NCH],
                                                 float (&dw)[NCH][kChunk]) {
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
  return dot;
}

// dx of a thread's columns; cd: dh (zeros without one).
template <bool BF16, int TPR, int NCH, bool STAGED>
__device__ __forceinline__ void backward_emit(const NormBackwardKernelArgs& a, int64_t base,
                                              bool live, int t, uint8_t* stage, float s,
                                              float mean, const Chunk<BF16> (&cy)[NCH],
                                              const Chunk<BF16> (&ch)[NCH],
                                              const Chunk<BF16> (&cd)[NCH]) {
  const int lane = threadIdx.x & 31;
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
      if (a.dh != nullptr) dx[i] = __fadd_rn(dx[i], cd[c].get(i));
    }
    Chunk<BF16> co;
    co.set(dx);
    co.store_warp<STAGED>(a.dx, base + col, n,
                          live ? warp_run(col - kChunk * lane, a.cols) : 0, a.g_dx, stage, lane);
  }
}

// One row of partial sums per CTA: its teams' dw in their order.
template <int TPR, int NCH>
__device__ __forceinline__ void backward_partials(const NormBackwardKernelArgs& a, int t,
                                                  int team, const float (&dw)[NCH][kChunk],
                                                  float* s_dw) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  constexpr int kTeams = kThreads / TPR;
  if (a.part == nullptr) return;
  float* out = a.part + (int64_t)blockIdx.x * a.cols;
  if constexpr (kTeams > 1) {
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
    for (int i = threadIdx.x; i < a.cols; i += kThreads) out[i] = s_dw[i];
  } else {
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int col = (c * TPR + t) * kChunk;
      Chunk<false> o;
      o.set(dw[c]);
      o.store(out, col, chunk_len(col, a.cols), a.g_part);
    }
  }
}

// CTA b takes the rows b, b + gridDim.x, ... (times its teams); each thread keeps the
// weight's gradient of its own columns in registers over all of them, so dw costs one
// row of partial sums per CTA.
template <bool BF16, int TPR, int NCH, bool STAGED>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
    k_add_rmsnorm_backward(const NormBackwardKernelArgs a) {
  // the columns' sum may be set up meanwhile; without one, the next launch in the stream is
  // another call's, which may count on this one's dx
  if (a.part != nullptr) pdl_launch_dependents();
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  constexpr int kTeams = kThreads / TPR;
  __shared__ float2 red[2][kThreads / 32];
  __shared__ float s_dw[kTeams > 1 ? TPR * NCH * kChunk : 1];
  __shared__ __align__(16) uint8_t stages[STAGED ? kThreads / 32 : 1][kStageBytes];
  const int t = threadIdx.x % TPR, team = threadIdx.x / TPR, lane = threadIdx.x & 31;
  uint8_t* stage = stages[STAGED ? threadIdx.x >> 5 : 0];
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
    Chunk<BF16> cy[NCH], ch[NCH], cd[NCH];
    {
      ChunkLoad<BF16, STAGED> ly[NCH], lh[NCH], ld[NCH];
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int col = (c * TPR + t) * kChunk;
        const int n = live ? chunk_len(col, a.cols) : 0;
        const int64_t run = live ? warp_run(col - kChunk * lane, a.cols) : 0;
        ly[c].issue(a.dy, base + col, n, run, a.g_dy, lane);
        lh[c].issue(a.h, base + col, n, run, a.g_h, lane);
        if (a.dh != nullptr) ld[c].issue(a.dh, base + col, n, run, a.g_dh, lane);
      }
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        cy[c] = ly[c].settle(a.g_dy, stage, lane);
        ch[c] = lh[c].settle(a.g_h, stage, lane);
        if (a.dh != nullptr) cd[c] = ld[c].settle(a.g_dh, stage, lane);
      }
    }
    const float dot = backward_gather<BF16, TPR, NCH>(a, t, s, cy, ch, dw);
    const float2 r = team_sum_max<TPR>(dot, 0.0f, red[buf]);
    backward_emit<BF16, TPR, NCH, STAGED>(a, base, live, t, stage, s, __fdiv_rn(r.x, (float)a.cols), cy, ch,
                                  cd);
  }
  backward_partials<TPR, NCH>(a, t, team, dw, s_dw);
}

// ANY: rows that are not 16-byte aligned (RowRing).
template <bool BF16, int TPR, int NCH, bool ANY>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
    k_add_rmsnorm_backward_ring(const NormBackwardKernelArgs a, const RingArgs g) {
  if (a.part != nullptr) pdl_launch_dependents();  // as above
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  constexpr int kTeams = kThreads / TPR;
  constexpr int kElem = BF16 ? 2 : 4;
  extern __shared__ __align__(128) uint8_t ring_smem[];
  __shared__ float2 red[2][kThreads / 32];
  __shared__ float s_dw[kTeams > 1 ? TPR * NCH * kChunk : 1];
  __shared__ __align__(8) uint64_t full[kRingStages];
  __shared__ int err;
  __shared__ __align__(16) uint8_t stages[ANY ? kThreads / 32 : 1][kStageBytes];
  uint8_t* out_stage = ANY ? stages[ANY ? threadIdx.x >> 5 : 0] : nullptr;
  const int t = threadIdx.x % TPR, team = threadIdx.x / TPR, lane = threadIdx.x & 31;
  const int64_t step = (int64_t)gridDim.x * kTeams;
  const RowRing<3, ANY> ring{full, &err, ring_smem, {a.dy, a.h, a.dh}, a.rows,
                             (int64_t)a.cols * kElem, kTeams, g};
  ring.start(step);
  float dw[NCH][kChunk];
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (int i = 0; i < kChunk; ++i) dw[c][i] = 0.0f;
  int it = 0, st = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * kTeams; row0 < a.rows; row0 += step, ++it) {
    const int64_t row = row0 + team;
    const bool live = row < a.rows;
    const float s = live ? a.rstd[row] : 0.0f;
    const uint8_t* p = ring.stage(st) + ring.shift(row0) + team * a.cols * kElem;
    const bool ok = ring.wait(st, it);
    ring.finish(st, row0);
    Chunk<BF16> cy[NCH], ch[NCH], cd[NCH];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int col = (c * TPR + t) * kChunk;
      const int n = live && ok ? chunk_len(col, a.cols) : 0;
      if constexpr (ANY) {
        const uint8_t* q = p + min(col, a.cols) * kElem;
        cy[c].load_shared_any(q, lane);
        ch[c].load_shared_any(q + g.tensor_bytes, lane);
        if (a.dh != nullptr) cd[c].load_shared_any(q + 2 * g.tensor_bytes, lane);
        cy[c].cut(n);
        ch[c].cut(n);
      } else {
        cy[c].load_shared(p + col * kElem, n, lane);
        ch[c].load_shared(p + g.tensor_bytes + col * kElem, n, lane);
        if (a.dh != nullptr) cd[c].load_shared(p + 2 * g.tensor_bytes + col * kElem, n, lane);
      }
    }
    const float dot = backward_gather<BF16, TPR, NCH>(a, t, s, cy, ch, dw);
    const float2 r = team_sum_max<TPR, true>(dot, 0.0f, red[it & 1]);
    if (*(volatile int*)&err) {
      ring.give_up(it, row0, step, a.status);
      return;
    }
    if (threadIdx.x == 0 && row0 + g.stages * step < a.rows)
      ring.fetch(st, row0 + g.stages * step);
    backward_emit<BF16, TPR, NCH, ANY>(a, row * a.cols, live, t, out_stage, s,
                                    __fdiv_rn(r.x, (float)a.cols), cy, ch, cd);
    if (++st == g.stages) st = 0;
  }
  backward_partials<TPR, NCH>(a, t, team, dw, s_dw);
}

// out[c] = sum over the n partial rows of part [n][cols], in a fixed order: warp w of a
// CTA adds the rows w, w + 8, ..., and the eight sums are added in turn.
__global__ void __launch_bounds__(256) k_column_sum(const float* part, int n, int64_t cols,
                                                    float* out) {
  __shared__ float s[8][32];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  float sum = 0.0f;
  if (col < cols)
#pragma unroll 4
    for (int r = warp; r < n; r += 8) sum = __fadd_rn(sum, part[(int64_t)r * cols + col]);
  s[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && col < cols) {
#pragma unroll
    for (int i = 1; i < 8; ++i) sum = __fadd_rn(sum, s[i][lane]);
    out[col] = sum;
  }
}

// The ring kernel, where at least two stages fit and every CTA has several groups (done).
template <bool BF16, int TPR, int NCH, bool ANY>
cudaError_t run_backward_ring(const NormBackwardKernelArgs& k, int64_t groups, int max_parts,
                              const DeviceInfo& dev, cudaStream_t stream, int* parts,
                              bool* done) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  auto ring = k_add_rmsnorm_backward_ring<BF16, TPR, NCH, ANY>;
  static const RingKernel limits = ring_kernel(ring, kThreads);
  const RingPlan p = plan_ring(limits, k.dh ? 3 : 2,
                               (int64_t)(kThreads / TPR) * k.cols * (BF16 ? 2 : 4), ANY);
  const int64_t fill = std::min<int64_t>((int64_t)p.ctas * dev.num_sms, max_parts);
  if (p.ctas == 0 || groups <= 2 * fill) return cudaSuccess;
  *done = true;
  const cudaError_t e = allow_ring(ring, limits);
  if (e != cudaSuccess) return e;
  *parts = (int)fill;
  ring<<<(unsigned)fill, kThreads, p.g.stages * p.g.stage_bytes, stream>>>(k, p.g);
  return cudaGetLastError();
}

template <bool BF16, int TPR, int NCH>
cudaError_t run_norm_backward(const NormBackwardKernelArgs& k, int max_parts,
                              const DeviceInfo& dev, cudaStream_t stream, int* parts) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  constexpr int kTeams = kThreads / TPR;
  const auto direct = k.g_min >= 16 ? k_add_rmsnorm_backward<BF16, TPR, NCH, false>
                                    : k_add_rmsnorm_backward<BF16, TPR, NCH, true>;
  static const int aligned = resident_ctas(k_add_rmsnorm_backward<BF16, TPR, NCH, false>, kThreads);
  static const int staged = resident_ctas(k_add_rmsnorm_backward<BF16, TPR, NCH, true>, kThreads);
  const int resident = k.g_min >= 16 ? aligned : staged;
  const int64_t groups = (k.rows + kTeams - 1) / kTeams;
  const int grid = (int)std::min<int64_t>(
      std::min<int64_t>(groups, (int64_t)resident * dev.num_sms), max_parts);
  bool done = false;
  cudaError_t e = cudaSuccess;
  if constexpr (BF16 || NCH == 1) {  // two stages of longer FP32 rows do not fit
    if (k.g_min >= 16)
      e = run_backward_ring<BF16, TPR, NCH, false>(k, groups, max_parts, dev, stream, parts, &done);
  }
  if constexpr (NCH == 1) {
    // Rows that are not aligned.  BF16, through the ring and loaded directly: 4000 x 5001 59
    // and 88 us, 16384 x 1001 46 and 76, 16384 x 25 30 and 35; FP32 4000 x 5001 74 and 123.
    if (k.g_min < 16 && k.bases_aligned)
      e = run_backward_ring<BF16, TPR, NCH, true>(k, groups, max_parts, dev, stream, parts, &done);
  }
  if (done || e != cudaSuccess) return e;
  *parts = grid;
  direct<<<grid, kThreads, 0, stream>>>(k);
  return cudaGetLastError();
}

template <bool BF16>
cudaError_t pick_norm_backward(const NormBackwardKernelArgs& k, int max_parts,
                               const DeviceInfo& dev, cudaStream_t stream, int* parts) {
  const int c = k.cols;
  if (c <= 512) return run_norm_backward<BF16, 32, 1>(k, max_parts, dev, stream, parts);
  if (c <= 1024) return run_norm_backward<BF16, 64, 1>(k, max_parts, dev, stream, parts);
  if (c <= 2048) return run_norm_backward<BF16, 128, 1>(k, max_parts, dev, stream, parts);
  if (c <= 4096) return run_norm_backward<BF16, 256, 1>(k, max_parts, dev, stream, parts);
  if (c <= 6144) return run_norm_backward<BF16, 384, 1>(k, max_parts, dev, stream, parts);
  if (c <= 8192) return run_norm_backward<BF16, 512, 1>(k, max_parts, dev, stream, parts);
  if (c <= 16384) return run_norm_backward<BF16, 1024, 1>(k, max_parts, dev, stream, parts);
  return run_norm_backward<BF16, 1024, 2>(k, max_parts, dev, stream, parts);
}

}  // namespace

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
  k.g_dy = row_grain(a.dy, a.cols * e);
  k.g_h = row_grain(a.h, a.cols * e);
  k.g_dh = row_grain(a.dh, a.cols * e);
  k.g_dx = row_grain(a.dx, a.cols * e);
  k.g_w = row_grain(a.weight, 0);
  k.g_part = row_grain(k.part, a.cols * 4);
  k.g_min = std::min(k.g_dy, std::min(k.g_h, k.g_dx));
  if (a.dh) k.g_min = std::min(k.g_min, k.g_dh);
  k.bases_aligned = (reinterpret_cast<uintptr_t>(a.dy) | reinterpret_cast<uintptr_t>(a.h) |
                     reinterpret_cast<uintptr_t>(a.dh)) % 16 == 0;
  k.status = dev.status;
  int parts = 0;
  const int max_parts = (int)std::min<int64_t>(a.rows, kNormBackwardParts);
  cudaError_t err = a.in == InType::BF16
                        ? pick_norm_backward<true>(k, max_parts, dev, stream, &parts)
                        : pick_norm_backward<false>(k, max_parts, dev, stream, &parts);
  if (err != cudaSuccess || a.dweight == nullptr) return err;
  return launch_after(k_column_sum, (unsigned)((a.cols + 31) / 32), 256, stream, (const float*)k.part,
                      parts, a.cols, a.dweight);
}

}  // namespace nvfp4
