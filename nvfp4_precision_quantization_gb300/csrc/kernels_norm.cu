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
  int* status;
};

constexpr float kE4m3Max = 448.0f;

// Encode scale of an E4M3 output whose largest magnitude is a.
__device__ __forceinline__ float fp8_encode_scale(float a) { return global_scale(a, kE4m3Max); }
__device__ __forceinline__ float fp8_decode_scale(float a) {
  return a == 0.0f ? 1.0f : fmaxf(__fdiv_rn(a, kE4m3Max), 0x1p-126f);
}

// Sum and maximum over the TPR threads of a row's team; every thread gets both.  The
// order of the sum depends on TPR alone.  red: one pair per warp, in two buffers used in
// turn, so that one barrier per row is enough.  BARRIER: with the CTA's barrier also where
// a team is one warp.
template <int TPR, bool BARRIER = false>
__device__ __forceinline__ float2 team_sum_max(float s, float m, float2* red) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, d));
    m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
  }
  if constexpr (TPR > 32) {
    constexpr int kWarps = TPR / 32;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) red[warp] = make_float2(s, m);
    __syncthreads();
    const float2 v = red[warp - warp % kWarps + lane % kWarps];
    s = v.x;
    m = v.y;
#pragma unroll
    for (int d = kWarps / 2; d > 0; d >>= 1) {
      s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, d));
      m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    }
  } else if constexpr (BARRIER) {
    __syncthreads();
  }
  return make_float2(s, m);
}

// What a thread does with its part of a row once h is in v: h out, then h w with the sum
// of h^2 and the maxima of |h w| (bmax per chunk).
template <bool BF16, int TPR, int NCH>
__device__ __forceinline__ void norm_gather(const NormKernelArgs& a, int64_t base, bool live, int t,
                                            float (&v)[NCH][kChunk], float (&bmax)[NCH],
                                            float& ss, float& mx) {
  ss = mx = 0.0f;
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
}

// The outputs of a row whose team found sum(h^2) = r.x and max|h w| = r.y.
template <bool BF16, bool NV4, int TPR, int NCH>
__device__ __forceinline__ void norm_emit(const NormKernelArgs& a, int64_t row, bool live, int t,
                                          float (&v)[NCH][kChunk], const float (&bmax)[NCH],
                                          float2 r) {
  const int64_t base = row * a.cols;
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

// Rows straight from memory into registers: few rows (each CTA has one or two, so there
// is nothing to run ahead of), and rows that are not 16-byte aligned.
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
    float v[NCH][kChunk], bmax[NCH], ss, mx;
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
    norm_gather<BF16, TPR, NCH>(a, base, live, t, v, bmax, ss, mx);
    const float2 r = team_sum_max<TPR>(ss, mx, red[buf]);
    norm_emit<BF16, NV4, TPR, NCH>(a, row, live, t, v, bmax, r);
  }
}

// ---------------------------------------------------------------- a ring of rows

// Many aligned rows: they run through a ring in shared memory, filled by bulk copies that
// thread 0 issues several rows ahead, so that the row's barrier and its arithmetic never
// leave the memory idle, whatever the registers allow to be resident.  A stage holds one
// group of kTeams consecutive rows of each tensor (consecutive in memory: one copy each).
// The row's reduction barrier is also what frees its stage: by then every thread has the
// stage's values in registers.
constexpr int kRingStages = 8;

struct RingArgs {
  int stages;
  int tensor_bytes;  // stride of a stage's tensors
  int stage_bytes;
};

template <int NT>
struct RowRing {
  uint64_t* full;
  int* err;
  uint8_t* smem;
  const void* src[NT];
  int64_t rows, row_bytes;
  int teams;
  RingArgs g;

  __device__ __forceinline__ uint8_t* stage(int s) const { return smem + s * g.stage_bytes; }
  // thread 0: start the copies of the group of rows that begins at row0
  __device__ __forceinline__ void fetch(int s, int64_t row0) const {
    const int64_t left = rows - row0;
    const uint32_t bytes = (uint32_t)((left < teams ? left : teams) * row_bytes);
    int n = 0;
#pragma unroll
    for (int i = 0; i < NT; ++i) n += src[i] != nullptr;
    mbar_expect_tx(&full[s], bytes * n);
#pragma unroll
    for (int i = 0; i < NT; ++i)
      if (src[i] != nullptr)
        bulk_copy_in(stage(s) + i * g.tensor_bytes,
                     static_cast<const char*>(src[i]) + row0 * row_bytes, bytes, &full[s]);
  }
  __device__ __forceinline__ void start(int64_t step) const {
    if (threadIdx.x == 0) {
      for (int s = 0; s < g.stages; ++s) mbar_init(&full[s], 1);
      *err = 0;
      fence_mbar_init();
      for (int s = 0; s < g.stages; ++s) {
        const int64_t row0 = (int64_t)blockIdx.x * teams + s * step;
        if (row0 < rows) fetch(s, row0);
      }
    }
    __syncthreads();
  }
  // Wait for use `it` of the ring; false (with the error noted) if it gave up.
  __device__ __forceinline__ bool wait(int s, int it) const {
    const bool ok = mbar_wait_bounded(&full[s], (it / g.stages) & 1);
    if (!ok) *err = 1;
    return ok;
  }
  // After a timeout: thread 0 waits (bounded) for the copies still in flight.
  __device__ __forceinline__ void give_up(int it, int64_t row0, int64_t step, int* status) const {
    if (threadIdx.x != 0) return;
    raise_status(status, kStatusTimeout);
    for (int k = 0; k < g.stages; ++k)
      if (row0 + k * step < rows)
        mbar_wait_bounded(&full[(it + k) % g.stages], ((it + k) / g.stages) & 1);
  }
};

template <bool BF16, bool NV4, int TPR, int NCH>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
    k_add_rmsnorm_ring(const NormKernelArgs a, const RingArgs g) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  constexpr int kTeams = kThreads / TPR;
  constexpr int kElem = BF16 ? 2 : 4;
  extern __shared__ __align__(128) uint8_t ring_smem[];
  __shared__ float2 red[2][kThreads / 32];
  __shared__ __align__(8) uint64_t full[kRingStages];
  __shared__ int err;
  const int t = threadIdx.x % TPR, team = threadIdx.x / TPR;
  const int64_t step = (int64_t)gridDim.x * kTeams;
  const RowRing<2> ring{full, &err, ring_smem, {a.x, a.res}, a.rows, (int64_t)a.cols * kElem,
                        kTeams, g};
  ring.start(step);
  int it = 0, s = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * kTeams; row0 < a.rows; row0 += step, ++it) {
    const int64_t row = row0 + team;
    const bool live = row < a.rows;
    const int64_t base = row * a.cols;
    const uint8_t* st = ring.stage(s) + team * a.cols * kElem;
    const bool ok = ring.wait(s, it);
    float v[NCH][kChunk], bmax[NCH], ss, mx;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int col = (c * TPR + t) * kChunk;
      const int n = live && ok ? chunk_len(col, a.cols) : 0;
      Chunk<BF16> cx;
      cx.load_shared(st + col * kElem, n, threadIdx.x & 31);
#pragma unroll
      for (int i = 0; i < kChunk; ++i) v[c][i] = cx.get(i);
      if (a.res != nullptr) {
        Chunk<BF16> cr;
        cr.load_shared(st + g.tensor_bytes + col * kElem, n, threadIdx.x & 31);
#pragma unroll
        for (int i = 0; i < kChunk; ++i) v[c][i] = __fadd_rn(v[c][i], cr.get(i));
      }
    }
    norm_gather<BF16, TPR, NCH>(a, base, live && ok, t, v, bmax, ss, mx);
    const float2 r = team_sum_max<TPR, true>(ss, mx, red[it & 1]);
    if (*(volatile int*)&err) {
      ring.give_up(it, row0, step, a.status);
      return;
    }
    if (threadIdx.x == 0 && row0 + g.stages * step < a.rows)
      ring.fetch(s, row0 + g.stages * step);
    norm_emit<BF16, NV4, TPR, NCH>(a, row, live, t, v, bmax, r);
    if (++s == g.stages) s = 0;
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
  int g_dy, g_h, g_dh, g_w, g_dx, g_part;
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
template <bool BF16, int TPR, int NCH>
__device__ __forceinline__ void backward_emit(const NormBackwardKernelArgs& a, int64_t base,
                                              bool live, int t, float s, float mean,
                                              const Chunk<BF16> (&cy)[NCH],
                                              const Chunk<BF16> (&ch)[NCH],
                                              const Chunk<BF16> (&cd)[NCH]) {
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
    co.store(a.dx, base + col, n, a.g_dx);
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
template <bool BF16, int TPR, int NCH>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
    k_add_rmsnorm_backward(const NormBackwardKernelArgs a) {
  pdl_launch_dependents();  // the columns' sum may be set up meanwhile
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
    Chunk<BF16> cy[NCH], ch[NCH], cd[NCH];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int col = (c * TPR + t) * kChunk;
      const int n = live ? chunk_len(col, a.cols) : 0;
      cy[c].load(a.dy, base + col, n, a.g_dy);
      ch[c].load(a.h, base + col, n, a.g_h);
      if (a.dh != nullptr) cd[c].load(a.dh, base + col, n, a.g_dh);
    }
    const float dot = backward_gather<BF16, TPR, NCH>(a, t, s, cy, ch, dw);
    const float2 r = team_sum_max<TPR>(dot, 0.0f, red[buf]);
    backward_emit<BF16, TPR, NCH>(a, base, live, t, s, __fdiv_rn(r.x, (float)a.cols), cy, ch, cd);
  }
  backward_partials<TPR, NCH>(a, t, team, dw, s_dw);
}

template <bool BF16, int TPR, int NCH>
__global__ void __launch_bounds__(TPR < 256 ? 256 : TPR)
    k_add_rmsnorm_backward_ring(const NormBackwardKernelArgs a, const RingArgs g) {
  pdl_launch_dependents();  // the columns' sum may be set up meanwhile
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  constexpr int kTeams = kThreads / TPR;
  constexpr int kElem = BF16 ? 2 : 4;
  extern __shared__ __align__(128) uint8_t ring_smem[];
  __shared__ float2 red[2][kThreads / 32];
  __shared__ float s_dw[kTeams > 1 ? TPR * NCH * kChunk : 1];
  __shared__ __align__(8) uint64_t full[kRingStages];
  __shared__ int err;
  const int t = threadIdx.x % TPR, team = threadIdx.x / TPR, lane = threadIdx.x & 31;
  const int64_t step = (int64_t)gridDim.x * kTeams;
  const RowRing<3> ring{full, &err, ring_smem, {a.dy, a.h, a.dh}, a.rows,
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
    const uint8_t* p = ring.stage(st) + team * a.cols * kElem;
    const bool ok = ring.wait(st, it);
    Chunk<BF16> cy[NCH], ch[NCH], cd[NCH];
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      const int col = (c * TPR + t) * kChunk;
      const int n = live && ok ? chunk_len(col, a.cols) : 0;
      cy[c].load_shared(p + col * kElem, n, lane);
      ch[c].load_shared(p + g.tensor_bytes + col * kElem, n, lane);
      if (a.dh != nullptr) cd[c].load_shared(p + 2 * g.tensor_bytes + col * kElem, n, lane);
    }
    const float dot = backward_gather<BF16, TPR, NCH>(a, t, s, cy, ch, dw);
    const float2 r = team_sum_max<TPR, true>(dot, 0.0f, red[it & 1]);
    if (*(volatile int*)&err) {
      ring.give_up(it, row0, step, a.status);
      return;
    }
    if (threadIdx.x == 0 && row0 + g.stages * step < a.rows)
      ring.fetch(st, row0 + g.stages * step);
    backward_emit<BF16, TPR, NCH>(a, row * a.cols, live, t, s, __fdiv_rn(r.x, (float)a.cols), cy,
                                  ch, cd);
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

template <typename K>
int resident_ctas(K kernel, int threads) {
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0) != cudaSuccess) {
    cudaGetLastError();
    n = 1;
  }
  return std::max(1, n);
}

// A ring kernel's CTAs per SM by registers, and its static shared memory.
constexpr int kCtaSmem = 227 << 10;  // shared memory that one CTA may have
struct RingKernel {
  int resident;
  int static_bytes;
};
template <typename K>
RingKernel ring_kernel(K kernel, int threads) {
  cudaFuncAttributes f;
  if (cudaFuncGetAttributes(&f, kernel) != cudaSuccess) {
    cudaGetLastError();
    return {0, 0};
  }
  return {resident_ctas(kernel, threads), (int)f.sharedSizeBytes};
}
template <typename K>
cudaError_t allow_ring(K kernel, const RingKernel& k) {  // on the current device
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              kCtaSmem - k.static_bytes);
}

// CTAs per SM and the ring of each: as many CTAs as the registers allow while each keeps
// at least two stages.  ctas == 0: two stages do not fit.
struct RingPlan {
  int ctas;
  RingArgs g;
};
RingPlan plan_ring(const RingKernel& k, int tensors, int64_t group_bytes) {
  RingPlan p{};
  const int64_t tensor = (group_bytes + 127) / 128 * 128, stage = tensors * tensor;
  for (int c = k.resident; c > 0; --c) {
    // an SM's 228 KB, of which every CTA takes 1 KB beside its own
    const int64_t room =
        std::min<int64_t>(kCtaSmem, (228 << 10) / c - (1 << 10)) - k.static_bytes;
    if (room < 2 * stage) continue;
    p.ctas = c;
    p.g.stages = (int)std::min<int64_t>(kRingStages, room / stage);
    p.g.tensor_bytes = (int)tensor;
    p.g.stage_bytes = (int)stage;
    break;
  }
  return p;
}

template <bool BF16, bool NV4, int TPR, int NCH>
cudaError_t run_norm(const NormKernelArgs& k, const DeviceInfo& dev, cudaStream_t stream) {
  constexpr int kThreads = TPR < 256 ? 256 : TPR;
  constexpr int kTeams = kThreads / TPR;
  static const int resident = resident_ctas(k_add_rmsnorm<BF16, NV4, TPR, NCH>, kThreads);
  const int64_t groups = (k.rows + kTeams - 1) / kTeams;
  const int64_t grid = std::min<int64_t>(groups, (int64_t)resident * dev.num_sms);
  if (k.g_x != 0 && (k.res == nullptr || k.g_res != 0)) {
    auto ring = k_add_rmsnorm_ring<BF16, NV4, TPR, NCH>;
    static const RingKernel limits = ring_kernel(ring, kThreads);
    const RingPlan p = plan_ring(limits, k.res ? 2 : 1,
                                 (int64_t)kTeams * k.cols * (BF16 ? 2 : 4));
    const int64_t fill = (int64_t)p.ctas * dev.num_sms;
    if (p.ctas > 0 && groups > 2 * fill) {
      const cudaError_t e = allow_ring(ring, limits);
      if (e != cudaSuccess) return e;
      ring<<<(unsigned)fill, kThreads, p.g.stages * p.g.stage_bytes, stream>>>(k, p.g);
      return cudaGetLastError();
    }
  }
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
  constexpr int kTeams = kThreads / TPR;
  static const int resident = resident_ctas(k_add_rmsnorm_backward<BF16, TPR, NCH>, kThreads);
  const int64_t groups = (k.rows + kTeams - 1) / kTeams;
  const int grid = (int)std::min<int64_t>(
      std::min<int64_t>(groups, (int64_t)resident * dev.num_sms), max_parts);
  if (k.g_dy != 0 && k.g_h != 0 && (k.dh == nullptr || k.g_dh != 0)) {
    auto ring = k_add_rmsnorm_backward_ring<BF16, TPR, NCH>;
    static const RingKernel limits = ring_kernel(ring, kThreads);
    const RingPlan p = plan_ring(limits, k.dh ? 3 : 2,
                                 (int64_t)kTeams * k.cols * (BF16 ? 2 : 4));
    const int64_t fill = std::min<int64_t>((int64_t)p.ctas * dev.num_sms, max_parts);
    if (p.ctas > 0 && groups > 2 * fill) {
      const cudaError_t e = allow_ring(ring, limits);
      if (e != cudaSuccess) return e;
      *parts = (int)fill;
      ring<<<(unsigned)fill, kThreads, p.g.stages * p.g.stage_bytes, stream>>>(k, p.g);
      return cudaGetLastError();
    }
  }
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
  return launch_after(k_column_sum, (unsigned)((cols + 31) / 32), 256, stream, part, n, cols, out);
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
  k.status = dev.status;
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
  k.g_part = row_grain(k.part, a.cols, 4);
  k.status = dev.status;
  int parts = 0;
  const int max_parts = (int)std::min<int64_t>(a.rows, kNormBackwardParts);
  cudaError_t err = a.in == InType::BF16
                        ? pick_norm_backward<true>(k, max_parts, dev, stream, &parts)
                        : pick_norm_backward<false>(k, max_parts, dev, stream, &parts);
  if (err != cudaSuccess || a.dweight == nullptr) return err;
  return launch_column_sum(k.part, parts, a.cols, a.dweight, stream);
}

}  // namespace nvfp4
