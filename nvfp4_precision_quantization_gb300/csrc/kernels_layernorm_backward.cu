// kernels_layernorm_backward.cu -- gradients of dropout, residual addition and layer norm.
//
//   dr = s (g - mean(g) - n mean(g n)) + dh,   n = (h - m) s,  g = dy w
//   dx = drop'(dr) (the forward's mask, made again),  dw = sum_rows dy n,  db = sum_rows dy
//
// Bound by memory: every tensor is read or written once.  A row's team of threads holds dy,
// h and dh in registers across the one reduction that the row needs (two sums), and each
// thread the parameters' gradients of its columns across all rows of its CTA, so they cost
// one row of partial sums per CTA, joined in a fixed order.
//
// Measured: 16384 x 8192 BF16 with dh 193 us, 5.6 TB/s, and with dropout (another tensor written) 256
// us, 5.2 TB/s (issue slots 48 % used by the 16 warps that the sums' registers leave an SM; bounded
// to 32 warps they spill, 298 us); 4000 x 5000 FP32 52 us, 4.6 TB/s, 43 without the parameters' gradients
// (their 12 MB of partial sums, written and read again, and the launch that joins them).  Rows of more
// than 8192 columns (1024 threads, 64 registers) and staged ones spill: 8000 x 12000 BF16 298 us for a
// floor of 141.
#include "dropout.cuh"
#include "row_ring.cuh"

namespace nvfp4 {
namespace {

struct LayerNormBackwardKernelArgs {
  const void* dy;
  const void* h;
  const void* dh;
  const void* w;
  const float* mean;
  const float* rstd;
  DropMask mask;
  void* dx;
  void* dres;   // or NULL
  float* part;  // [gridDim.x][2][cols] partial dweight and dbias, or NULL
  int64_t rows;
  int cols;
  bool w_bf16;
  int g_dy, g_h, g_dh, g_w, g_dx, g_dres, g_part;
  int g_min;  // the least of those of dy, h, dh, dx and dres
  bool bases_aligned;  // dy, h and dh start on 16 bytes
  int* status;
};

template <bool BF16>
__device__ __forceinline__ Pair chunk_pair(const Chunk<BF16>& c, int i) {
  return {c.get(2 * i), c.get(2 * i + 1)};
}

// The parameters' gradients of a thread's columns over its rows, two columns at a time.
template <int NCH>
struct ParamSums {
  Pair w[NCH][kChunk / 2], b[NCH][kChunk / 2];
  __device__ __forceinline__ ParamSums() {
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int i = 0; i < kChunk / 2; ++i) w[c][i] = b[c][i] = {0.0f, 0.0f};
  }
};

// What a row's values become, kept across its reduction: n = (h - m) s and g = dy w.
template <int NCH>
struct RowTerms {
  Pair n[NCH][kChunk / 2], g[NCH][kChunk / 2];
};

// Adds 16 columns of a row to a thread's sums of the parameters' gradients (w, b) and of the row's
// g and g n (total, dot); wc: the weights.
template <bool BF16, bool WEIGHT_BF16>
__device__ __forceinline__ void gather16(const Chunk<WEIGHT_BF16>& wc, float m, float s,
                                         const Chunk<BF16>& cy, const Chunk<BF16>& ch,
                                         Pair (&n)[kChunk / 2], Pair (&g)[kChunk / 2],
                                         Pair (&w)[kChunk / 2], Pair (&b)[kChunk / 2], Pair& total,
                                         Pair& dot) {
#pragma unroll
  for (int i = 0; i < kChunk / 2; ++i) {
    const Pair dy = chunk_pair(cy, i);
    n[i] = pair_mul(pair_add(chunk_pair(ch, i), {-m, -m}), {s, s});
    g[i] = pair_mul(dy, chunk_pair(wc, i));
    w[i] = pair_fma(dy, n[i], w[i]);
    b[i] = pair_add(dy, b[i]);
    total = pair_add(total, g[i]);
    dot = pair_fma(g[i], n[i], dot);
  }
}

// Adds a row to a thread's sums; the row's own sums of g and g n of those columns.
template <bool BF16, int TPR, int NCH>
__device__ __forceinline__ float2 backward_gather(const LayerNormBackwardKernelArgs& a, int t,
                                                  float m, float s, const Chunk<BF16> (&cy)[NCH],
                                                  const Chunk<BF16> (&ch)[NCH],
                                                  RowTerms<NCH>& terms, ParamSums<NCH>& sums) {
  Pair total = {0.0f, 0.0f}, dot = {0.0f, 0.0f};
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int col = (c * TPR + t) * kChunk, n = chunk_len(col, a.cols);
    if (a.w_bf16) {
      Chunk<true> w;
      w.load(a.w, col, n, a.g_w);
      gather16(w, m, s, cy[c], ch[c], terms.n[c], terms.g[c], sums.w[c], sums.b[c], total, dot);
    } else {
      Chunk<false> w;
      w.load(a.w, col, n, a.g_w);
      gather16(w, m, s, cy[c], ch[c], terms.n[c], terms.g[c], sums.w[c], sums.b[c], total, dot);
    }
  }
  return make_float2(__fadd_rn(total.x, total.y), __fadd_rn(dot.x, dot.y));
}

// dr and dx of a thread's columns; mg, mgn: the row's means; cd: dh (unused without one).
template <bool BF16, int TPR, int NCH, bool STAGED>
__device__ __forceinline__ void backward_emit(const LayerNormBackwardKernelArgs& a,
                                              const Dropper& drop, int64_t base, bool live, int t,
                                              uint8_t* stage, float s, float mg, float mgn,
                                              const RowTerms<NCH>& terms,
                                              const Chunk<BF16> (&cd)[NCH]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int col = (c * TPR + t) * kChunk;
    const int n = live ? chunk_len(col, a.cols) : 0;
    const int64_t run = live ? warp_run(col - kChunk * lane, a.cols) : 0;
    float d[kChunk];
#pragma unroll
    for (int i = 0; i < kChunk / 2; ++i) {
      Pair g = pair_fma(terms.n[c][i], {-mgn, -mgn}, pair_add(terms.g[c][i], {-mg, -mg}));
      g = a.dh != nullptr ? pair_fma(g, {s, s}, chunk_pair(cd[c], i)) : pair_mul(g, {s, s});
      d[2 * i] = g.x;
      d[2 * i + 1] = g.y;
    }
    Chunk<BF16> co;
    if (a.dres != nullptr) {
      co.set(d);
      co.template store_warp<STAGED>(a.dres, base + col, n, run, a.g_dres, stage, lane);
    }
    drop.apply<BF16>(base + col, d, nullptr);
    co.set(d);
    co.template store_warp<STAGED>(a.dx, base + col, n, run, a.g_dx, stage, lane);
  }
}

// One row of partial sums per CTA: its teams' in their order.
template <int TPR, int NCH>
__device__ __forceinline__ void backward_partials(const LayerNormBackwardKernelArgs& a, int t,
                                                  int team, const ParamSums<NCH>& sums,
                                                  float* s_sum) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  constexpr int kTeams = kThreads / TPR;
  if (a.part == nullptr) return;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* out = a.part + ((int64_t)blockIdx.x * 2 + which) * a.cols;
    const auto& from = which == 0 ? sums.w : sums.b;
    if constexpr (kTeams > 1) {
      for (int k = 0; k < kTeams; ++k) {
        if (team == k) {
#pragma unroll
          for (int c = 0; c < NCH; ++c)
#pragma unroll
            for (int i = 0; i < kChunk; ++i) {
              float* p = &s_sum[(c * TPR + t) * kChunk + i];
              const float v = (i & 1) ? from[c][i / 2].y : from[c][i / 2].x;
              *p = k == 0 ? v : __fadd_rn(*p, v);
            }
        }
        __syncthreads();
      }
      for (int i = threadIdx.x; i < a.cols; i += kThreads) out[i] = s_sum[i];
      __syncthreads();
    } else {
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        const int col = (c * TPR + t) * kChunk;
        Chunk<false> o;
#pragma unroll
        for (int i = 0; i < kChunk; ++i)
          o.w[i] = __float_as_uint((i & 1) ? from[c][i / 2].y : from[c][i / 2].x);
        o.store(out, col, chunk_len(col, a.cols), a.g_part);
      }
    }
  }
}

// Sums over a team, of both at once (red as in team_sum_max).
template <int TPR, bool BARRIER>
__device__ __forceinline__ float2 team_sum2(float2 v, float2* red) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    v.x = __fadd_rn(v.x, __shfl_xor_sync(0xffffffffu, v.x, d));
    v.y = __fadd_rn(v.y, __shfl_xor_sync(0xffffffffu, v.y, d));
  }
  if constexpr (TPR > 32) {
    constexpr int kWarps = TPR / 32;
    constexpr int kTree = kWarps <= 2 ? 2 : kWarps <= 4 ? 4 : kWarps <= 8 ? 8 : kWarps <= 16 ? 16 : 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    const int i = lane % kTree;
    v = i < kWarps ? red[warp - warp % kWarps + i] : make_float2(0.0f, 0.0f);
#pragma unroll
    for (int d = kTree / 2; d > 0; d >>= 1) {
      v.x = __fadd_rn(v.x, __shfl_xor_sync(0xffffffffu, v.x, d));
      v.y = __fadd_rn(v.y, __shfl_xor_sync(0xffffffffu, v.y, d));
    }
  } else if constexpr (BARRIER) {
    __syncthreads();
  }
  return v;
}

// CTA b takes the rows b, b + gridDim.x, ... (times its teams).
template <bool BF16, int TPR, int NCH, bool STAGED>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
    k_layernorm_backward(const LayerNormBackwardKernelArgs a) {
  // the columns' sum may be set up meanwhile; without one, the next launch in the stream is
  // another call's, which may count on this one's dx
  if (a.part != nullptr) pdl_launch_dependents();
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  constexpr int kTeams = kThreads / TPR;
  __shared__ float2 red[2][kThreads / 32];
  __shared__ float s_sum[kTeams > 1 ? TPR * NCH * kChunk : 1];
  __shared__ __align__(16) uint8_t stages[STAGED ? kThreads / 32 : 1][kStageBytes];
  const int t = threadIdx.x % TPR, team = threadIdx.x / TPR, lane = threadIdx.x & 31;
  uint8_t* stage = stages[STAGED ? threadIdx.x >> 5 : 0];
  const Dropper drop(a.mask);
  ParamSums<NCH> sums;
  const float inv_cols = __frcp_rn((float)a.cols);
  int buf = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * kTeams; row0 < a.rows;
       row0 += (int64_t)gridDim.x * kTeams, buf ^= 1) {
    const int64_t row = row0 + team;
    const bool live = kTeams == 1 || row < a.rows;
    const int64_t base = row * a.cols;
    const float m = live ? a.mean[row] : 0.0f, s = live ? a.rstd[row] : 0.0f;
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
    RowTerms<NCH> terms;
    float2 r = backward_gather<BF16, TPR, NCH>(a, t, m, s, cy, ch, terms, sums);
    r = team_sum2<TPR, false>(r, red[buf]);
    backward_emit<BF16, TPR, NCH, STAGED>(a, drop, base, live, t, stage, s,
                                          __fmul_rn(r.x, inv_cols), __fmul_rn(r.y, inv_cols),
                                          terms, cd);
  }
  backward_partials<TPR, NCH>(a, t, team, sums, s_sum);
}

// CTAs per SM that the registers have to allow: two of up to 320 threads, one of more (bounded to
// 24 warps a row's accumulators spill).
constexpr int backward_ctas(int threads) { return threads <= 320 ? 2 : 1; }

// Many rows through a shared-memory ring.  ANY: rows that are not 16-byte aligned (RowRing).
template <bool BF16, int TPR, int NCH, bool ANY>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR, backward_ctas(TPR))
    k_layernorm_backward_ring(const LayerNormBackwardKernelArgs a, const RingArgs g) {
  if (a.part != nullptr) pdl_launch_dependents();  // as above
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  constexpr int kTeams = kThreads / TPR;
  constexpr int kElem = BF16 ? 2 : 4;
  extern __shared__ __align__(128) uint8_t ring_smem[];
  __shared__ float2 red[2][kThreads / 32];
  __shared__ float s_sum[kTeams > 1 ? TPR * NCH * kChunk : 1];
  __shared__ __align__(8) uint64_t full[kRingStages];
  __shared__ int err;
  __shared__ __align__(16) uint8_t stages[ANY ? kThreads / 32 : 1][kStageBytes];
  uint8_t* out_stage = ANY ? stages[ANY ? threadIdx.x >> 5 : 0] : nullptr;
  const int t = threadIdx.x % TPR, team = threadIdx.x / TPR, lane = threadIdx.x & 31;
  const int64_t step = (int64_t)gridDim.x * kTeams;
  const RowRing<3, ANY> ring{full, &err, ring_smem, {a.dy, a.h, a.dh}, a.rows,
                             (int64_t)a.cols * kElem, kTeams, g};
  const Dropper drop(a.mask);
  ring.start(step);
  ParamSums<NCH> sums;
  const float inv_cols = __frcp_rn((float)a.cols);
  int it = 0, st = 0;
  // a row's statistics are loaded a row ahead: nothing else of it comes from far
  float next_m = 0.0f, next_s = 0.0f;
  auto fetch = [&](int64_t row) {
    if (row < a.rows) next_m = a.mean[row], next_s = a.rstd[row];
  };
  fetch((int64_t)blockIdx.x * kTeams + team);
  for (int64_t row0 = (int64_t)blockIdx.x * kTeams; row0 < a.rows; row0 += step, ++it) {
    const int64_t row = row0 + team;
    const bool live = kTeams == 1 || row < a.rows;
    const float m = live ? next_m : 0.0f, s = live ? next_s : 0.0f;
    fetch(row + step);
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
    RowTerms<NCH> terms;
    float2 r = backward_gather<BF16, TPR, NCH>(a, t, m, s, cy, ch, terms, sums);
    r = team_sum2<TPR, true>(r, red[it & 1]);
    if (*(volatile int*)&err) {
      ring.give_up(it, row0, step, a.status);
      return;
    }
    if (threadIdx.x == 0 && row0 + g.stages * step < a.rows)
      ring.fetch(st, row0 + g.stages * step);
    backward_emit<BF16, TPR, NCH, ANY>(a, drop, row * a.cols, live, t, out_stage, s,
                                       __fmul_rn(r.x, inv_cols), __fmul_rn(r.y, inv_cols), terms,
                                       cd);
    if (++st == g.stages) st = 0;
  }
  backward_partials<TPR, NCH>(a, t, team, sums, s_sum);
}

// dweight and dbias [cols] from n rows of part [n][2][cols], in a fixed order: warp w of a CTA
// adds the rows w, w + 8, ..., and the eight sums are added in turn.
__global__ void __launch_bounds__(256) k_param_sums(const float* part, int n, int64_t cols,
                                                    float* dweight, float* dbias) {
  __shared__ float s[8][32];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + lane;
  float sum = 0.0f;
  if (col < 2 * cols)
#pragma unroll 4
    for (int r = warp; r < n; r += 8) sum = __fadd_rn(sum, part[(int64_t)r * 2 * cols + col]);
  s[warp][lane] = sum;
  __syncthreads();
  if (warp == 0 && col < 2 * cols) {
#pragma unroll
    for (int i = 1; i < 8; ++i) sum = __fadd_rn(sum, s[i][lane]);
    float* out = col < cols ? dweight : dbias;
    if (out != nullptr) out[col < cols ? col : col - cols] = sum;
  }
}

// The ring kernel, where at least two stages fit and every CTA has several groups (done).
template <bool BF16, int TPR, int NCH, bool ANY>
cudaError_t run_ring(const LayerNormBackwardKernelArgs& k, int64_t groups, int max_parts,
                     const DeviceInfo& dev, cudaStream_t stream, int* parts, bool* done) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  auto ring = k_layernorm_backward_ring<BF16, TPR, NCH, ANY>;
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
cudaError_t run(const LayerNormBackwardKernelArgs& k, int max_parts, const DeviceInfo& dev,
                cudaStream_t stream, int* parts) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  constexpr int kTeams = kThreads / TPR;
  const auto direct = k.g_min >= 16 ? k_layernorm_backward<BF16, TPR, NCH, false>
                                    : k_layernorm_backward<BF16, TPR, NCH, true>;
  static const int aligned = resident_ctas(k_layernorm_backward<BF16, TPR, NCH, false>, kThreads);
  static const int staged = resident_ctas(k_layernorm_backward<BF16, TPR, NCH, true>, kThreads);
  const int resident = k.g_min >= 16 ? aligned : staged;
  const int64_t groups = (k.rows + kTeams - 1) / kTeams;
  const int grid = (int)std::min<int64_t>(
      std::min<int64_t>(groups, (int64_t)resident * dev.num_sms), max_parts);
  bool done = false;
  cudaError_t e = cudaSuccess;
  if constexpr (BF16 || NCH == 1) {  // two stages of longer FP32 rows do not fit
    if (k.g_min >= 16)
      e = run_ring<BF16, TPR, NCH, false>(k, groups, max_parts, dev, stream, parts, &done);
  }
  if constexpr (NCH == 1) {
    if (k.g_min < 16 && k.bases_aligned)
      e = run_ring<BF16, TPR, NCH, true>(k, groups, max_parts, dev, stream, parts, &done);
  }
  if (done || e != cudaSuccess) return e;
  *parts = grid;
  direct<<<grid, kThreads, 0, stream>>>(k);
  return cudaGetLastError();
}

template <bool BF16>
cudaError_t pick(const LayerNormBackwardKernelArgs& k, int max_parts, const DeviceInfo& dev,
                 cudaStream_t stream, int* parts) {
  const int c = k.cols;
  if (c <= 512) return run<BF16, 32, 1>(k, max_parts, dev, stream, parts);
  if (c <= 1024) return run<BF16, 64, 1>(k, max_parts, dev, stream, parts);
  if (c <= 2048) return run<BF16, 128, 1>(k, max_parts, dev, stream, parts);
  if (c <= 4096) return run<BF16, 256, 1>(k, max_parts, dev, stream, parts);
  if (c <= 5120) return run<BF16, 320, 1>(k, max_parts, dev, stream, parts);
  if (c <= 6144) return run<BF16, 384, 1>(k, max_parts, dev, stream, parts);
  if (c <= 8192) return run<BF16, 512, 1>(k, max_parts, dev, stream, parts);
  if (c <= 16384) return run<BF16, 1024, 1>(k, max_parts, dev, stream, parts);
  return run<BF16, 1024, 2>(k, max_parts, dev, stream, parts);
}

}  // namespace

int64_t add_layernorm_backward_workspace(int64_t rows, int64_t cols) {
  // one row of partial sums per CTA; no more CTAs than kLayerNormBackwardParts, nor than rows
  return 8 * cols * std::min<int64_t>(rows, kLayerNormBackwardParts);
}

cudaError_t launch_add_layernorm_backward(const NormBackwardArgs& a, const DeviceInfo& dev,
                                          cudaStream_t stream) {
  if (a.cols == 0) return cudaSuccess;
  if (a.rows == 0) {
    cudaError_t e = cudaSuccess;
    if (a.dweight) e = cudaMemsetAsync(a.dweight, 0, 4 * a.cols, stream);
    if (e == cudaSuccess && a.dbias) e = cudaMemsetAsync(a.dbias, 0, 4 * a.cols, stream);
    return e;
  }
  const int e = a.in == InType::BF16 ? 2 : 4;
  LayerNormBackwardKernelArgs k{};
  k.dy = a.dy;
  k.h = a.h;
  k.dh = a.dh;
  k.w = a.weight;
  k.mean = a.mean;
  k.rstd = a.rstd;
  k.mask = a.mask;
  k.dx = a.dx;
  k.dres = a.dresidual;
  k.part = a.dweight || a.dbias ? static_cast<float*>(a.workspace) : nullptr;
  k.rows = a.rows;
  k.cols = (int)a.cols;
  k.w_bf16 = a.weight_bf16;
  k.g_dy = row_grain(a.dy, a.cols * e);
  k.g_h = row_grain(a.h, a.cols * e);
  k.g_dh = row_grain(a.dh, a.cols * e);
  k.g_dx = row_grain(a.dx, a.cols * e);
  k.g_dres = row_grain(a.dresidual, a.cols * e);
  k.g_w = row_grain(a.weight, 0);
  k.g_part = row_grain(k.part, a.cols * 4);
  k.g_min = std::min(k.g_dy, std::min(k.g_h, k.g_dx));
  if (a.dh) k.g_min = std::min(k.g_min, k.g_dh);
  if (a.dresidual) k.g_min = std::min(k.g_min, k.g_dres);
  k.bases_aligned = (reinterpret_cast<uintptr_t>(a.dy) | reinterpret_cast<uintptr_t>(a.h) |
                     reinterpret_cast<uintptr_t>(a.dh)) % 16 == 0;
  k.status = dev.status;
  int parts = 0;
  const int max_parts = (int)std::min<int64_t>(a.rows, kLayerNormBackwardParts);
  cudaError_t err = a.in == InType::BF16 ? pick<true>(k, max_parts, dev, stream, &parts)
                                         : pick<false>(k, max_parts, dev, stream, &parts);
  if (err != cudaSuccess || k.part == nullptr) return err;
  return launch_after(k_param_sums, (unsigned)((2 * a.cols + 31) / 32), 256, stream,
                      (const float*)k.part, parts, a.cols, a.dweight, a.dbias);
}

}  // namespace nvfp4
