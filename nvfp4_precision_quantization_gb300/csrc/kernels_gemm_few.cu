// kernels_gemm_few.cu -- the NVFP4 product with its epilogue for few rows of A (decoded
// tokens, short prompts): D [m][n] = act(A B^T + bias) + residual.
//
// With few rows the product reads B (the weights) once and is bound by that: 0.5625 bytes
// per weight.  So the roles are exchanged: 128 lines of B are the MMA's M, up to 64 rows
// of A (padded to 16, 32 or 64) its N, and what has to be right is the stream of B:
//   * every SM's CTA streams tiles of 128 lines (and up to 64 rows) through K in units of
//     512 values; the tiles that do not go round are cut along K (plan_cut), so that all SMs
//     stream to the end.  The parts of a tile are joined by the CTA that finishes it last,
//     from partial sums in the workspace, added in their order (the result does not depend
//     on which CTA that is);
//   * the compact scales are read as they lie (no pass over them beforehand), kGroup units
//     of a line at a time (16 bytes of a line alone would fetch a 64-byte burst for each
//     unit): asynchronous copies to shared memory a group ahead, from there to registers
//     and into tensor memory.
// GATED (the gated product, D = act(A Bg^T + bg) (A Bu^T + bu), B's lines the gate's and then
// the up projection's): a tile is 128 lines of each, in two accumulators, so that a lane of the
// epilogue holds both factors of its column; a unit is 256 values of the 256 lines.
// Warps: 0 loads codes (TMA, a ring of S stages), 1 issues the MMAs, 2-5 copy scales and
// write them to TMEM (one per lane quarter), 6-9 are the epilogue (two accumulators, so the
// next tile's MMAs run meanwhile).  Lane l of the accumulator is line l of B, so a warp
// writes 32 neighbouring columns of D for each row.
//
// Measured (bias, GELU): one row times 28672 x 8192 weights 26 us, 5.1 TB/s (launch, first
// loads and the last epilogue are about 6 us of it), times 114688 x 8192 80 us, 6.6 TB/s, 0.98
// of a copy; 300 rows times 2048 x 7168 16 us, and 20 with a residual.  GATED (SiLU): one row times 2 x
// 28672 x 8192 46 us, 5.7 TB/s.
//
// Every wait is bounded, as in kernels_gemm.cu; a tile's partial sums are never waited
// for: whoever arrives last has them.
#include <algorithm>

#include "activation.cuh"
#include "internal.h"
#include "row_io.cuh"
#include "tcgen05.cuh"

namespace nvfp4 {
namespace {

constexpr int kLines = 128;     // lines of B per tile = MMA M
constexpr int kBoxBytes = 128;  // code bytes of a line per TMA box: 256 values
// Boxes of B per unit, eight MMAs: 512 values of 128 lines, or (GATED) 256 values of 128 lines
// of either half of B.  (One box a unit measured 0.42 us a unit on rows where memory does not
// bound, most of it the waits and issues of single threads.)
constexpr int kBoxes = 2;
template <bool GATED>
struct Unit {
  static constexpr int kHalves = GATED ? 2 : 1;       // of B, an accumulator each
  static constexpr int kKBoxes = kBoxes / kHalves;    // along K
  static constexpr int kBytes = kKBoxes * kBoxBytes;  // of a line
  static constexpr int kScales = kBytes / 8;
  static constexpr int kSteps = kBytes / 32;          // MMAs along K, 64 values each
  static constexpr int kSlotCols = (kHalves + 1) * 4 * kSteps;  // TMEM columns of a unit's
                                                                // scales: B's halves, A's
};
constexpr int kEpiWarps = 4;     // one per TMEM lane quarter
constexpr int kFewThreads = 32 * (6 + kEpiWarps);
constexpr int kMaxCtas = 160;   // bound of the grid, for the workspace

struct FewParams {
  const uint8_t* x_scales;
  const uint8_t* w_scales;
  int x_grain, w_grain;  // how the scale rows are copied: 16, 2 or 1 (see copy_lines)
  const float* x_amax;
  const float* w_amax;
  int x_amax_stride, w_amax_stride;
  float x_finv, w_finv;
  int m, n;
  int64_t k16;      // scales per line
  int k_tiles;      // units per tile
  int m_tiles;      // tiles along A's rows, side by side for each 128 lines of B
  int tiles;        // all tiles
  int split, parts; // the first `split` tiles are cut into `parts` along K
  void* d;
  bool d_bf16;
  Epilogue epi;
  GatedOut gated;      // GATED
  uint32_t* arrivals;  // [split], zero before the kernel's first arrival
  float4* sums;        // [split][parts][halves][NT / 4][128] partial sums, four rows of A each
  uint32_t idesc;
  int* status;
};

// Scales of a group of kGroup units, one row of shared memory per line.  The pitch is an
// odd number of 16-byte units, so lanes reading their own lines meet no bank conflict.
template <int kGroup, bool GATED>
struct ScaleRows {
  static constexpr int kRowBytes = kGroup * Unit<GATED>::kScales;
  static constexpr int kPitch = kRowBytes + 16;
};

// 16 bytes, of which those from `bytes` on become zero and are not read.
__device__ __forceinline__ void cp_async16(void* dst, const void* src, int bytes = 16) {
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)),
               "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void cp_async_wait_all() {
  asm volatile("cp.async.wait_all;" ::: "memory");
}

// Start copying bytes [b0, b0 + kRowBytes) of the scale rows [first, first + lines) of
// sc [total][k16] (rows from total on are left alone) to rows of dst; t of 128 threads.
//   grain 16: rows and base are 16-byte aligned; 2: the base is, and the 16-byte units that
//   cover a row's part are copied, so that it starts 0 to 14 bytes (k16 is even) into its row
//   of dst; no byte outside the tensor is read; 1: bytes, not asynchronously.
template <class ROWS>
__device__ __forceinline__ void copy_lines(const uint8_t* sc, int64_t k16, int64_t total,
                                           int64_t first, int lines, int64_t b0, int grain,
                                           uint8_t* dst, int t) {
  constexpr int kRow = ROWS::kRowBytes, kPitch = ROWS::kPitch;
  const int bytes = (int)min((int64_t)kRow, k16 - b0);
  const int rows = (int)min((int64_t)lines, total - first);
  // four warps issue this between units: pointers step by constants, nothing is divided
  if (grain == 16) {
    constexpr int kParts = kRow / 16, kStep = 128 / kParts;  // rows side by side
    const int c = 16 * (t % kParts);
    if (c >= bytes) return;
    const uint8_t* from = sc + (first + t / kParts) * k16 + b0 + c;
    dst += t / kParts * kPitch + c;
#pragma unroll 4
    for (int r = t / kParts; r < rows; r += kStep, from += kStep * k16, dst += kStep * kPitch)
      cp_async16(dst, from);
  } else if (grain == 2) {
    const int64_t end = total * k16;
    for (int r = t; r < rows; r += 128) {
      const int64_t from = (first + r) * k16 + b0, to = from + bytes;
      int64_t at = from & ~(int64_t)15;
      uint8_t* row = dst + r * kPitch;
#pragma unroll
      for (int c = 0; c <= kRow / 16; ++c, at += 16, row += 16)
        if (at < to) cp_async16(row, sc + at, (int)min((int64_t)16, end - at));
    }
  } else {
    for (int i = t; i < rows * kRow; i += 128) {
      const int r = i / kRow, c = i % kRow;
      if (c < bytes) dst[r * kPitch + c] = sc[(first + r) * k16 + b0 + c];
    }
  }
}

// The scales of unit e of the group, of the line at src, as words (one per MMA); those from n
// on zero (they belong to the next line).  shift: where in its first 16 bytes the row starts.
template <int kMmas>
__device__ __forceinline__ void read_scales(const uint8_t* src, int e, int shift, int n,
                                            uint32_t* w) {
  constexpr int kUnitScales = 4 * kMmas;
  const uint8_t* p = src + kUnitScales * e;
  if (shift == 0) {
#pragma unroll
    for (int j = 0; j < kMmas; j += 4) {
      const uint4 v = *reinterpret_cast<const uint4*>(p + 4 * j);
      w[j] = v.x, w[j + 1] = v.y, w[j + 2] = v.z, w[j + 3] = v.w;
    }
  } else {
    const uint32_t* q = reinterpret_cast<const uint32_t*>(p + (shift & ~3));
    uint32_t v[kMmas + 1];
#pragma unroll
    for (int j = 0; j < kMmas; ++j) v[j] = q[j];
    v[kMmas] = (shift & 2) ? q[kMmas] : 0u;
#pragma unroll
    for (int j = 0; j < kMmas; ++j) w[j] = __funnelshift_r(v[j], v[j + 1], 8 * (shift & 2));
  }
  if (n < kUnitScales) {
#pragma unroll
    for (int j = 0; j < kMmas; ++j) {
      const int left = n - 4 * j;
      if (left <= 0) w[j] = 0;
      else if (left < 4) w[j] &= (1u << (8 * left)) - 1u;
    }
  }
}

// Named barrier over THREADS threads, with the OR of a flag: 1 the epilogue's, 2 the scales'.
template <int ID, int THREADS>
__device__ __forceinline__ bool barrier_or(bool flag) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"((uint32_t)flag), "n"(ID), "n"(THREADS)
      : "memory");
  return any != 0;
}

// A CTA's walk, segment by segment.  The first p.split tiles are cut along K into p.parts
// parts each, and the parts dealt to the CTAs in turn; the tiles after them (a whole number
// for every CTA) are taken whole, and last, so that the joining of the parts happens while
// they stream.
struct Walk {
  int part;  // the next part
  int next;  // the next whole tile
  int tile, slice, kt, kt1;  // the segment: units [kt, kt1) of the tile, its part `slice`
  __device__ __forceinline__ Walk(const FewParams& p)
      : part(blockIdx.x), next(p.split + blockIdx.x) {}
  __device__ __forceinline__ bool advance(const FewParams& p) {
    if (part < p.split * p.parts) {
      tile = part / p.parts;
      slice = part % p.parts;
      part += gridDim.x;
      kt = p.k_tiles * slice / p.parts;
      kt1 = p.k_tiles * (slice + 1) / p.parts;
      return true;
    }
    if (next >= p.tiles) return false;
    tile = next;
    next += gridDim.x;
    kt = 0;
    kt1 = p.k_tiles;
    return true;
  }
};

// The residual of rows row .. row + R - 1 of one column (nothing without one).
template <int R>
__device__ __forceinline__ void few_residual(const FewParams& p, int row, int col, float* r) {
  if (p.epi.residual == nullptr) return;
  const int64_t at = (int64_t)row * p.n + col;
  const int rows = p.m - row;
  if (p.d_bf16) {
    const __nv_bfloat16* from = static_cast<const __nv_bfloat16*>(p.epi.residual) + at;
#pragma unroll
    for (int j = 0; j < R; ++j)
      if (j < rows) r[j] = __bfloat162float(from[(int64_t)j * p.n]);
  } else {
    const float* from = static_cast<const float*>(p.epi.residual) + at;
#pragma unroll
    for (int j = 0; j < R; ++j)
      if (j < rows) r[j] = from[(int64_t)j * p.n];
  }
}

// Rows row .. row + R - 1 of one column: the scaled sums v (as in kernels_gemm.cu), the
// epilogue with the residual r, the stores.  alpha: the row factors in shared memory.
template <int R>
__device__ __forceinline__ void few_store(const FewParams& p, int row, int col, float* v,
                                          const float* r, const float* alpha, float beta,
                                          float bias) {
#pragma unroll
  for (int j = 0; j < R; ++j)
    v[j] = __fadd_rn(__fmul_rn(__fmul_rn(v[j], alpha[j]), beta), bias);
  const int64_t at = (int64_t)row * p.n + col;
  const int rows = p.m - row;
  auto store = [&](void* base) {
    if (p.d_bf16) {
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(base) + at;
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (j < rows) o[(int64_t)j * p.n] = __float2bfloat16_rn(v[j]);
    } else {
      float* o = static_cast<float*>(base) + at;
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (j < rows) o[(int64_t)j * p.n] = v[j];
    }
  };
  if (p.epi.z != nullptr) store(p.epi.z);
  apply_act<R>(p.epi.act, v);
  if (p.epi.residual != nullptr) {
#pragma unroll
    for (int j = 0; j < R; ++j)
      if (j < rows) v[j] = __fadd_rn(v[j], r[j]);
  }
  store(p.d);
}

// NT: rows of A per MMA (its N); S: stages of the code ring and of the TMEM scale slots;
// kGroup: units per scale copy (two groups in shared memory).
template <int NT, int S, int kGroup, bool GATED>
struct FewGeom {
  using U = Unit<GATED>;
  static constexpr int kABytes = kLines * kBoxes * kBoxBytes;
  static constexpr int kStageBytes = kABytes + NT * U::kBytes;
  // (32 rows at least: every lane reads one)
  static constexpr int kScaleBytes =
      (U::kHalves * kLines + (NT < 32 ? 32 : NT)) * ScaleRows<kGroup, GATED>::kPitch;
  static constexpr int kSmemBytes =
      S * kStageBytes + 2 * kScaleBytes + 512 /* barriers */ + 1024 /* alignment */;
  // two accumulators (of each half), then the scale slots
  static constexpr int kSfCol0 = 2 * U::kHalves * NT;
  static constexpr int kTmemCols = 512;
  static_assert(kSfCol0 + U::kSlotCols * S <= kTmemCols, "TMEM columns");
  static_assert(kStageBytes % 1024 == 0, "128B swizzle");
  static_assert(kScaleBytes % 16 == 0, "16-byte rows");
  static_assert(kSmemBytes + kEpiWarps * NT * 4 <= 232448, "shared memory");
};

// Rows row .. row + R - 1 of one column (live: there is one) of the gated product: g and u the
// scaled sums of its halves, d = act(g) u; cmax, the column's maximum of |d| as stored, grows.
template <int R>
__device__ __forceinline__ void few_store_gated(const FewParams& p, int row, int col, bool live,
                                                float* g, float* u, const float* alpha,
                                                const float (&beta)[2], const float (&bias)[2],
                                                float& cmax, int lane) {
  static_assert(R == 16, "the reduction below is of 16 rows");
#pragma unroll
  for (int j = 0; j < R; ++j) {
    g[j] = __fadd_rn(__fmul_rn(__fmul_rn(g[j], alpha[j]), beta[0]), bias[0]);
    u[j] = __fadd_rn(__fmul_rn(__fmul_rn(u[j], alpha[j]), beta[1]), bias[1]);
  }
  const int rows = live ? p.m - row : 0;
  auto store = [&](void* base, int64_t at, int64_t pitch, const float* v) {
    if (p.d_bf16) {
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(base) + at;
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (j < rows) o[(int64_t)j * pitch] = __float2bfloat16_rn(v[j]);
    } else {
      float* o = static_cast<float*>(base) + at;
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (j < rows) o[(int64_t)j * pitch] = v[j];
    }
  };
  if (p.gated.gu != nullptr) {
    const int64_t at = (int64_t)row * 2 * p.n + col;
    store(p.gated.gu, at, 2 * (int64_t)p.n, g);
    store(p.gated.gu, at + p.n, 2 * (int64_t)p.n, u);
  }
  apply_act<R>(p.epi.act, g);
#pragma unroll
  for (int j = 0; j < R; ++j) g[j] = __fmul_rn(g[j], u[j]);
  store(p.d, (int64_t)row * p.n + col, p.n, g);
  if (p.gated.row_amax == nullptr && p.gated.col_amax == nullptr) return;
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const float as = p.d_bf16 ? __bfloat162float(__float2bfloat16_rn(g[j])) : g[j];
    g[j] = j < rows ? fmaxf(fabsf(as), 0.0f) : 0.0f;  // NaN skipped
    cmax = fmaxf(cmax, g[j]);
  }
  if (p.gated.row_amax == nullptr) return;
  // the rows' maxima over the lanes: half of the rows go with each step, so lane l ends with row
  // l / 2
#pragma unroll
  for (int d = 16, n = R / 2; n > 0; d >>= 1, n >>= 1) {
    const bool upper = lane & d;
#pragma unroll
    for (int j = 0; j < n; ++j) {
      const float give = upper ? g[j] : g[j + n], keep = upper ? g[j + n] : g[j];
      g[j] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, d));
    }
  }
  g[0] = fmaxf(g[0], __shfl_xor_sync(0xffffffffu, g[0], 1));
  // non-negative floats are ordered like their bits, and a maximum does not depend on its order
  const int at = row + (lane >> 1);
  if (!(lane & 1) && at < p.m)
    atomicMax(reinterpret_cast<int*>(p.gated.row_amax) + at, __float_as_int(g[0]));
}

template <int NT, int S, int kGroup, bool GATED>
__global__ void __launch_bounds__(kFewThreads, 1)
    k_gemm_few(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
               const FewParams p) {
  using G = FewGeom<NT, S, kGroup, GATED>;
  using U = Unit<GATED>;
  using Rows = ScaleRows<kGroup, GATED>;
  constexpr int kSteps = U::kSteps;
  constexpr int kXGroups = (NT + 31) / 32;  // 32-row groups of A: TMEM columns of its scales
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* scale_smem = smem + S * G::kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(scale_smem + 2 * G::kScaleBytes);
  uint64_t* empty = full + S;
  uint64_t* sf_full = empty + S;
  uint64_t* acc_full = sf_full + S;
  uint64_t* acc_empty = acc_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  int* err = reinterpret_cast<int*>(tmem_slot + 1);
  int* last_flag = err + 1;
  __shared__ float s_alpha[kEpiWarps][NT];  // each epilogue warp's row factors

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&sf_full[s], 4);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], kEpiWarps);
    }
    *err = 0;
    fence_mbar_init();
    prefetch_tmap(&map_w);
    prefetch_tmap(&map_x);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, G::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0 && lane == 0) {
    // ---------------- codes
    const uint64_t pol_w = policy_evict_normal(), pol_x = policy_evict_last();
    uint32_t it = 0;
    bool ok = true;
    for (Walk w(p); ok && w.advance(p);) {
      const int line0 = w.tile / p.m_tiles * kLines, row0 = w.tile % p.m_tiles * NT;
      for (int kt = w.kt; kt < w.kt1; ++kt, ++it) {
        const uint32_t s = it % S;
        if (it >= (uint32_t)S && !mbar_wait_bounded(&empty[s], ((it / S) - 1) & 1)) *err = 1;
        if (*(volatile int*)err) {
          ok = false;
          break;
        }
        uint8_t* st = smem + s * G::kStageBytes;
        mbar_expect_tx(&full[s], G::kStageBytes);
#pragma unroll
        for (int b = 0; b < kBoxes; ++b) {  // a box past K is all zeros
          const int x = kt * U::kBytes + b % U::kKBoxes * kBoxBytes;
          const int line = line0 + b / U::kKBoxes * p.n;
          tma_load_2d(st + b * kLines * kBoxBytes, &map_w, &full[s], x, line, pol_w);
          if (b < U::kKBoxes)
            tma_load_2d(st + G::kABytes + b * NT * kBoxBytes, &map_x, &full[s], x, row0, pol_x);
        }
      }
    }
    // every copy issued must have landed before the CTA may exit
    for (uint32_t j = it > (uint32_t)S ? it - S : 0; j < it; ++j)
      if (!mbar_wait_bounded(&full[j % S], (j / S) & 1)) *err = 1;
  } else if (warp == 1 && lane == 0) {
    // ---------------- MMAs: one accumulator per segment
    uint32_t it = 0, seg = 0;
    bool ok = true;
    for (Walk w(p); ok && w.advance(p); ++seg) {
      const uint32_t b = seg & 1;
      if (seg >= 2 && !mbar_wait_bounded(&acc_empty[b], ((seg >> 1) - 1) & 1)) {
        *err = 1;
        break;
      }
      tc_fence_after();
      for (int kt = w.kt; kt < w.kt1; ++kt, ++it) {
        const uint32_t s = it % S, ph = (it / S) & 1;
        if (!mbar_wait_bounded(&sf_full[s], ph) || !mbar_wait_bounded(&full[s], ph)) {
          *err = 1;
          ok = false;
          break;
        }
        if (*(volatile int*)err) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t st = smem_addr(smem + s * G::kStageBytes);
        const uint32_t sf = tmem + G::kSfCol0 + U::kSlotCols * s;
#pragma unroll
        for (int i = 0; i < U::kHalves * kSteps; ++i) {
          const int ks = i / U::kHalves, half = i % U::kHalves;
          const int box = ks / 4, at = 32 * (ks % 4);
          tc_mma_nvf4(tmem + (b * U::kHalves + half) * NT,
                      desc_swz128(st + (half * U::kKBoxes + box) * kLines * kBoxBytes + at),
                      desc_swz128(st + G::kABytes + box * NT * kBoxBytes + at), p.idesc,
                      sf + 4 * (half * kSteps + ks), sf + 4 * (U::kHalves * kSteps + ks),
                      kt != w.kt || ks != 0);
        }
        tc_commit(&empty[s]);
      }
      tc_commit(&acc_full[b]);
    }
    // everything issued must be done before TMEM is freed
    for (uint32_t j = seg > 2 ? seg - 2 : 0; j < seg; ++j)
      if (!mbar_wait_bounded(&acc_full[j & 1], (j >> 1) & 1)) *err = 1;
  } else if (warp >= 2 && warp < 6) {
    // ---------------- scales: lane quarter q holds the B lines 32q + lane, and a copy of
    // the scales of the tile's rows of A
    const int q = warp & 3, t = threadIdx.x - 64;
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    constexpr int kPitch = Rows::kPitch, kBLines = U::kHalves * kLines;
    auto copy = [&](const Walk& w, int kt, int slot) {
      const int64_t b0 = (int64_t)(kt / kGroup) * Rows::kRowBytes;
      uint8_t* dst = scale_smem + slot * G::kScaleBytes;
#pragma unroll
      for (int h = 0; h < U::kHalves; ++h)
        copy_lines<Rows>(p.w_scales, p.k16, (int64_t)(h + 1) * p.n,
                         (int64_t)h * p.n + (int64_t)(w.tile / p.m_tiles) * kLines, kLines, b0,
                         p.w_grain, dst + h * kLines * kPitch, t);
      copy_lines<Rows>(p.x_scales, p.k16, p.m, (int64_t)(w.tile % p.m_tiles) * NT, NT, b0,
                       p.x_grain, dst + kBLines * kPitch, t);
    };
    // `w` walks the copies, one group of units ahead of those written to TMEM
    Walk w(p);
    bool more = w.advance(p), ok = true;
    int next_kt = w.kt;
    if (more) copy(w, next_kt, 0);
    uint32_t it = 0;
    for (int slot = 0; more; slot ^= 1) {
      // this group has arrived, and everyone is done with the one before it
      cp_async_wait_all();
      if (barrier_or<2, 128>(!ok || *(volatile int*)err)) {
        *err = 1;
        break;
      }
      const int tile = w.tile;
      int kt = next_kt;
      const int end = min(w.kt1, (kt / kGroup + 1) * kGroup);
      next_kt = end;
      if (end == w.kt1) {
        more = w.advance(p);
        next_kt = w.kt;
      }
      if (more) copy(w, next_kt, slot ^ 1);
      const int64_t line = (int64_t)(tile / p.m_tiles) * kLines + 32 * q + lane;
      const int64_t row = (int64_t)(tile % p.m_tiles) * NT + lane;
      const uint8_t* w_row = scale_smem + slot * G::kScaleBytes + (32 * q + lane) * kPitch;
      const uint8_t* x_row = scale_smem + slot * G::kScaleBytes + (kBLines + lane) * kPitch;
      // a row's part starts where the row does, 16 bytes times a whole number further on
      int w_shift[U::kHalves];
#pragma unroll
      for (int h = 0; h < U::kHalves; ++h)
        w_shift[h] = p.w_grain == 2 ? (int)(((line + (int64_t)h * p.n) * p.k16) & 15) : 0;
      for (; kt < end; ++kt, ++it) {
        const int e = kt % kGroup;
        const int n = (int)min((int64_t)U::kScales, p.k16 - (int64_t)kt * U::kScales);
        uint32_t wa[U::kHalves][kSteps], wb[kXGroups][kSteps];
#pragma unroll
        for (int h = 0; h < U::kHalves; ++h)
          read_scales<kSteps>(w_row + h * kLines * kPitch, e, w_shift[h], n, wa[h]);
#pragma unroll
        for (int c = 0; c < kXGroups; ++c)
          read_scales<kSteps>(x_row + (NT >= 32 ? 32 * c : 0) * kPitch, e,
                              p.x_grain == 2 ? (int)(((row + 32 * c) * p.k16) & 15) : 0, n, wb[c]);
        const uint32_t st = it % S;
        if (ok && it >= (uint32_t)S) ok = mbar_wait_bounded(&empty[st], ((it / S) - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) continue;  // to the group's end, where the four warps leave together
        tc_fence_after();
        const uint32_t sf = tmem + lanes + G::kSfCol0 + U::kSlotCols * st;
#pragma unroll
        for (int m = 0; m < kSteps; m += 4) {
          uint32_t r[16];
#pragma unroll
          for (int h = 0; h < U::kHalves; ++h) {
#pragma unroll
            for (int k = 0; k < 16; ++k) r[k] = wa[h][m + (k >> 2)];  // read at column q of each four
            tmem_st16(sf + 4 * (h * kSteps + m), r);
          }
#pragma unroll
          for (int k = 0; k < 16; ++k)
            r[k] = (k & 3) < kXGroups ? wb[(k & 3) < kXGroups ? (k & 3) : 0][m + (k >> 2)] : 0u;
          tmem_st16(sf + 4 * (U::kHalves * kSteps + m), r);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sf_full[st]);
      }
    }
    cp_async_wait_all();
  } else if (warp >= 6) {
    // ---------------- epilogue
    const int q = warp & 3, l = 32 * q + lane;
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    uint32_t seg = 0;
    for (Walk w(p); w.advance(p); ++seg) {
      const int tile = w.tile;
      const bool whole = w.kt == 0 && w.kt1 == p.k_tiles;
      const uint32_t b = seg & 1;
      const int col = tile / p.m_tiles * kLines + l;
      const int row0 = tile % p.m_tiles * NT, rows = min(NT, p.m - row0);
      const bool live = col < p.n;
      float* alpha = s_alpha[warp - 6];
      __syncwarp();  // every lane is done with the previous tile's factors
      for (int j = lane; j < NT; j += 32)
        alpha[j] = j < rows ? __fmul_rn(__ldg(p.x_amax + (int64_t)(row0 + j) * p.x_amax_stride),
                                        p.x_finv)
                            : 0.0f;
      __syncwarp();
      float beta[U::kHalves], bias[U::kHalves], cmax = 0.0f;
#pragma unroll
      for (int h = 0; h < U::kHalves; ++h) {
        beta[h] = bias[h] = 0.0f;
        if (live) {
          const int line = col + h * p.n;
          beta[h] = __fmul_rn(__ldg(p.w_amax + (int64_t)line * p.w_amax_stride), p.w_finv);
          bias[h] = p.epi.bias_at(line);
        }
      }
      // the residual is loaded 16 rows ahead of its use, the first before the sums are ready
      // (not for a part: whoever joins the tile may be writing d, which may be the residual)
      float r[16];
      if (!GATED && live && whole) few_residual<16>(p, row0, col, r);
      const bool ready = mbar_wait_bounded(&acc_full[b], (seg >> 1) & 1);
      if (!ready) *err = 1;
      if (barrier_or<1, 32 * kEpiWarps>(!ready || *(volatile int*)err)) break;
      tc_fence_after();
      if constexpr (GATED) {
        if (p.gated.row_amax != nullptr || p.gated.col_amax != nullptr) pdl_wait();  // are zero
      }
      constexpr int64_t kHalfSums = (NT / 4) * kLines;
      constexpr int64_t kSums = U::kHalves * kHalfSums;  // of one part
      float4* part = p.sums + ((int64_t)tile * p.parts + w.slice) * kSums + l;
#pragma unroll 1
      for (int c = 0; c < rows; c += 16) {
        float next[16];
        if (!GATED && whole && live && c + 16 < rows)
          few_residual<16>(p, row0 + c + 16, col, next);
        uint32_t v[U::kHalves][16];
#pragma unroll
        for (int h = 0; h < U::kHalves; ++h)
          tmem_ld16(tmem + lanes + (b * U::kHalves + h) * NT + c, v[h]);
        tmem_ld_wait();
        float f[U::kHalves][16];
#pragma unroll
        for (int h = 0; h < U::kHalves; ++h)
#pragma unroll
          for (int j = 0; j < 16; ++j) f[h][j] = __uint_as_float(v[h][j]);
        if (!whole) {
#pragma unroll
          for (int h = 0; h < U::kHalves; ++h)
#pragma unroll
            for (int g = 0; g < 4; ++g)
              if (c + 4 * g < rows)
                __stcg(part + h * kHalfSums + (c / 4 + g) * kLines,
                       make_float4(f[h][4 * g], f[h][4 * g + 1], f[h][4 * g + 2], f[h][4 * g + 3]));
        } else if constexpr (GATED) {
          few_store_gated<16>(p, row0 + c, col, live, f[0], f[1], alpha + c, beta, bias, cmax, lane);
        } else if (live) {
          few_store<16>(p, row0 + c, col, f[0], r, alpha + c, beta[0], bias[0]);
#pragma unroll
          for (int j = 0; j < 16; ++j) r[j] = next[j];
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[b]);
      // the column's maximum, once its tile is whole
      auto store_cmax = [&] {
        if (GATED && live && p.gated.col_amax != nullptr)
          atomicMax(reinterpret_cast<int*>(p.gated.col_amax) + col, __float_as_int(cmax));
      };
      if (whole) {
        store_cmax();
        continue;
      }
      // the CTA that finishes the tile last adds its parts, in their order
      barrier_or<1, 32 * kEpiWarps>(false);  // the four warps' sums are written (and released below)
      if (warp == 6 && lane == 0) {
        pdl_wait();  // the arrival counts are zero
        __threadfence();
        *last_flag = atomicAdd(p.arrivals + tile, 1u) == (uint32_t)(p.parts - 1);
        __threadfence();
      }
      barrier_or<1, 32 * kEpiWarps>(false);
      const bool last = *(volatile int*)last_flag != 0;
      barrier_or<1, 32 * kEpiWarps>(false);  // read before it is written again
      if (!last || (!GATED && !live)) continue;
      const int groups = (rows + 3) / 4;
      if constexpr (!GATED) few_residual<16>(p, row0, col, r);
      const float4* from = p.sums + (int64_t)tile * p.parts * kSums + l;
#pragma unroll 1
      for (int g0 = 0; g0 < groups; g0 += 4) {
        float next[16], fs[U::kHalves][16];
        if (!GATED && g0 + 4 < groups) few_residual<16>(p, row0 + 4 * g0 + 16, col, next);
#pragma unroll
        for (int h = 0; h < U::kHalves; ++h) {
          float* f = fs[h];
          auto load = [&](int part, float4 (&a)[4]) {
#pragma unroll
            for (int g = 0; g < 4; ++g)
              if (g0 + g < groups)
                a[g] = __ldcg(from + part * kSums + h * kHalfSums + (g0 + g) * kLines);
          };
#pragma unroll
          for (int j = 0; j < 16; ++j) f[j] = 0.0f;
          // three parts in flight at a time
#pragma unroll 1
          for (int c = 0; c < p.parts; c += 3) {
            float4 a[3][4];
#pragma unroll
            for (int k = 0; k < 3; ++k)
              if (c + k < p.parts) load(c + k, a[k]);
#pragma unroll
            for (int k = 0; k < 3; ++k)
#pragma unroll
              for (int g = 0; g < 4; ++g)
                if (c + k < p.parts && g0 + g < groups) {
                  f[4 * g] = __fadd_rn(f[4 * g], a[k][g].x);
                  f[4 * g + 1] = __fadd_rn(f[4 * g + 1], a[k][g].y);
                  f[4 * g + 2] = __fadd_rn(f[4 * g + 2], a[k][g].z);
                  f[4 * g + 3] = __fadd_rn(f[4 * g + 3], a[k][g].w);
                }
          }
        }
        if constexpr (GATED) {
          few_store_gated<16>(p, row0 + 4 * g0, col, live, fs[0], fs[1], alpha + 4 * g0, beta, bias,
                              cmax, lane);
        } else {
          few_store<16>(p, row0 + 4 * g0, col, fs[0], r, alpha + 4 * g0, beta[0], bias[0]);
#pragma unroll
          for (int j = 0; j < 16; ++j) r[j] = next[j];
        }
      }
      store_cmax();
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *(volatile int*)err) raise_status(p.status, kStatusTimeout);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, G::kTmemCols);
  }
}

// Clears the arrival counts, and the maxima that the product raises.  The product starts while
// this runs (it needs them only at its first shared tile or its first result).
struct ClearArgs {
  void* p[3];
  int n[3];  // words
};
__global__ void __launch_bounds__(256) k_clear_words(const ClearArgs a) {
  pdl_launch_dependents();
#pragma unroll
  for (int k = 0; k < 3; ++k)
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.n[k];
         i += (int64_t)gridDim.x * 256)  // (a count near 2^31 leaves no room for an int's last step)
      static_cast<uint32_t*>(a.p[k])[i] = 0;
}
cudaError_t launch_clear(const ClearArgs& a, cudaStream_t stream) {
  const int64_t words = (int64_t)a.n[0] + a.n[1] + a.n[2];
  k_clear_words<<<(unsigned)std::min<int64_t>((words + 1023) / 1024, 64), 256, 0, stream>>>(a);
  return cudaGetLastError();
}

// The gated product of an empty sum (k == 0): every row is act(bias_g) bias_u.
__global__ void __launch_bounds__(256) k_gated_epilogue_only(const Epilogue e, const GatedOut o,
                                                             void* d, bool bf16, int64_t m, int n) {
  auto put = [&](void* base, int64_t i, float v) {
    if (bf16) static_cast<__nv_bfloat16*>(base)[i] = __float2bfloat16_rn(v);
    else static_cast<float*>(base)[i] = v;
  };
  const int64_t total = m * n;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
       i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / n;
    const int c = (int)(i % n);
    float v[2] = {e.bias_at(c), 0.0f};
    const float u = e.bias_at(n + c);
    if (o.gu != nullptr) {
      put(o.gu, 2 * r * n + c, v[0]);
      put(o.gu, (2 * r + 1) * n + c, u);
    }
    apply_act<2>(e.act, v);
    const float z = __fmul_rn(v[0], u);
    put(d, i, z);
    const float as = bf16 ? __bfloat162float(__float2bfloat16_rn(z)) : z;
    const int top = __float_as_int(fmaxf(fabsf(as), 0.0f));
    if (o.row_amax != nullptr) atomicMax(reinterpret_cast<int*>(o.row_amax) + r, top);
    if (o.col_amax != nullptr) atomicMax(reinterpret_cast<int*>(o.col_amax) + c, top);
  }
}

int scale_grain(const uint8_t* p, int64_t k16) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return (a | (uintptr_t)k16) % 16 == 0 ? 16 : (a % 16 == 0 ? 2 : 1);
}

int rows_of_mma(int64_t m) { return m <= 16 ? 16 : (m <= 32 ? 32 : 64); }
int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t tiles_of(int64_t m, int64_t n) {
  return ceil_div(n, kLines) * ceil_div(m, rows_of_mma(m));
}
int64_t round256(int64_t v) { return (v + 255) / 256 * 256; }

// How many tiles are cut along K, and into how many parts.  `sms` CTAs take tiles / sms
// whole tiles each; the rest is cut where that is faster.  In nanoseconds: a unit takes
// about 500 for a CTA alone and 840 when every SM streams (memory); joining adds about 4000
// at the end of the call (two passes through L2 and their fences), nothing where whole
// tiles follow.  (Measured on the product without a gate; a GATED unit has as many bytes and MMAs.)
struct CutPlan {
  int split, parts;
};
CutPlan plan_cut(int tiles, int k_tiles, int sms) {
  CutPlan best{tiles % sms, 1};
  int64_t best_ns = INT64_MAX;
  const int rest = tiles % sms;
  for (int parts = 1; rest > 0 && parts <= 8 && 2 * parts <= std::max(2, k_tiles); ++parts) {
    const int64_t all = (int64_t)rest * parts;
    if (parts > 1 && all > 2 * kMaxCtas) break;  // what the workspace holds
    const int64_t active = std::min<int64_t>(all, sms), rounds = (all + sms - 1) / sms;
    const int64_t unit = std::max<int64_t>(500, 840 * active / sms);
    const int64_t ns = rounds * ((k_tiles + parts - 1) / parts) * unit +
                       (parts > 1 && tiles < sms ? 4000 : 0);
    if (ns < best_ns) {
      best_ns = ns;
      best.parts = parts;
    }
  }
  return best;
}

template <int NT, int S, int kGroup, bool GATED>
cudaError_t run_few(FewParams& p, const CUtensorMap& map_w, const CUtensorMap& map_x, int grid,
                    cudaStream_t stream) {
  using G = FewGeom<NT, S, kGroup, GATED>;
  auto kernel = k_gemm_few<NT, S, kGroup, GATED>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       G::kSmemBytes);
  if (e != cudaSuccess) return e;
  p.idesc = make_idesc_nvf4(kLines, NT);
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = G::kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  const ClearArgs clear{{p.arrivals, p.gated.row_amax, p.gated.col_amax},
                        {p.parts > 1 ? p.split : 0, p.gated.row_amax ? p.m : 0,
                         p.gated.col_amax ? p.n : 0}};
  if (clear.n[0] > 0 || clear.n[1] > 0 || clear.n[2] > 0) {
    if ((e = launch_clear(clear, stream)) != cudaSuccess) return e;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, kernel, map_w, map_x, p);
}

}  // namespace

cudaError_t launch_gated_epilogue_only(const Epilogue& e, const GatedOut& g, void* d, bool bf16,
                                       int64_t m, int64_t n, const DeviceInfo& dev,
                                       cudaStream_t stream) {
  const int64_t grid = std::min<int64_t>((m * n + 255) / 256, 8LL * dev.num_sms);
  const ClearArgs clear{{nullptr, g.row_amax, g.col_amax},
                        {0, g.row_amax ? (int)m : 0, g.col_amax ? (int)n : 0}};
  if (clear.n[1] > 0 || clear.n[2] > 0) {
    const cudaError_t err = launch_clear(clear, stream);
    if (err != cudaSuccess) return err;
  }
  k_gated_epilogue_only<<<(unsigned)grid, 256, 0, stream>>>(e, g, d, bf16, m, (int)n);
  return cudaGetLastError();
}

// Up to 384 rows, or up to 304 tiles (two for each of 152 SMs).  Measured with bias and GELU,
// this kernel against k_gemm_nvf4, in us: (m, n, k) = (64, 8192, 8192) 19 and 43, (384, 8192,
// 8192) 40 and 45, (384, 28672, 8192) 101 and 108; beyond, (512, 8192, 8192) 47 and 46, (512,
// 28672, 8192) 132 and 109, (1024, 8192, 8192) 81 and 65; but with few tiles (512, 2048,
// 7168) 18 and 31, (512, 4096, 4096) 21 and 26, (1000, 1024, 4096) 14 and 25.
bool gemm_few(int64_t m, int64_t n) { return m <= 384 || tiles_of(m, n) <= 304; }

// Up to one MMA's rows; up to a tile a CTA of short sums, where the other kernel's pre-pass is
// what counts; and, in up to two rounds of the other kernel, rows of D that are not 16-byte
// aligned, which its epilogue has to transpose.  This kernel and k_gemm_gated, in us: (m, n, k) =
// (1, 28672, 8192) 48 and 84, (64, 14336, 8192) 30 and 42; (64, 8192, 8192) 28 and 26, (128, 14336,
// 8192) 41 and 43, (256, 8192, 8192) 49 and 28; (256, 1024, 1024) 8.8 and 10.2, (256, 2048, 2048)
// 11.8 both, (2048, 1024, 1024) 14.8 and 11.6; unaligned (500, 1001, 1024) 8.9 and 13.7, (300,
// 5001, 7168) 37 and 41, (2000, 5001, 2048) 63 and 51.  One border for all lengths gives 2 us away on either
// side of it, at (64, 8192, 8192) and (128, 14336, 8192).
bool gemm_gated_few(int64_t m, int64_t n, int64_t k, bool aligned) {
  return m <= 64 || (k <= 1024 && tiles_of(m, n) <= 152) ||
         (!aligned && ceil_div(m, 256) * ceil_div(n, 128) <= 152);
}

int64_t gemm_few_workspace(int64_t m, int64_t n, bool gated) {
  return round256(4 * tiles_of(m, n)) +
         (int64_t)(gated ? 2 : 1) * kMaxCtas * 2 * rows_of_mma(m) * kLines * 4;
}

cudaError_t launch_gemm_few(const GemmArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  const int nt = rows_of_mma(a.M);
  const bool gated = a.gated != nullptr;
  CUtensorMap map_w, map_x;
  if (!make_operand_map(&map_w, a.b_codes, gated ? 2 * a.N : a.N, a.K / 2, kBoxBytes, kLines) ||
      !make_operand_map(&map_x, a.a_codes, a.M, a.K / 2, kBoxBytes, nt))
    return cudaErrorInvalidValue;
  FewParams p{};
  p.x_scales = a.a_scales;
  p.w_scales = a.b_scales;
  p.k16 = a.K / 16;
  p.x_grain = scale_grain(a.a_scales, p.k16);
  p.w_grain = scale_grain(a.b_scales, p.k16);
  p.x_amax = a.a_amax;
  p.w_amax = a.b_amax;
  p.x_amax_stride = a.a_row_scaled ? 1 : 0;
  p.w_amax_stride = a.b_row_scaled ? 1 : 0;
  p.x_finv = 1.0f / (a.a_bound * 6.0f);
  p.w_finv = 1.0f / (a.b_bound * 6.0f);
  p.m = (int)a.M;
  p.n = (int)a.N;
  const int64_t unit = 2 * (gated ? Unit<true>::kBytes : Unit<false>::kBytes);  // values
  p.k_tiles = (int)ceil_div(a.K, unit);
  p.m_tiles = (int)ceil_div(a.M, nt);
  p.tiles = (int)tiles_of(a.M, a.N);
  p.d = a.d;
  p.d_bf16 = a.d_bf16;
  p.epi = *a.epilogue;
  if (gated) p.gated = *a.gated;
  p.arrivals = reinterpret_cast<uint32_t*>(a.workspace);
  p.sums = reinterpret_cast<float4*>(a.workspace + round256(4 * (int64_t)p.tiles));
  p.status = dev.status;
  const int grid = std::min(p.tiles, std::min(dev.num_sms, kMaxCtas));
  const CutPlan cut = plan_cut(p.tiles, p.k_tiles, std::min(dev.num_sms, kMaxCtas));
  p.split = cut.split;
  p.parts = cut.parts;
  const int ctas = std::max(grid, std::min(std::min(dev.num_sms, kMaxCtas), p.split * p.parts));
  if (gated) {
    switch (nt) {
      case 16: return run_few<16, 4, 8, true>(p, map_w, map_x, ctas, stream);
      case 32: return run_few<32, 4, 4, true>(p, map_w, map_x, ctas, stream);
      default: return run_few<64, 4, 4, true>(p, map_w, map_x, ctas, stream);
    }
  }
  switch (nt) {
    case 16: return run_few<16, 4, 4, false>(p, map_w, map_x, ctas, stream);
    case 32: return run_few<32, 4, 4, false>(p, map_w, map_x, ctas, stream);
    default: return run_few<64, 3, 4, false>(p, map_w, map_x, ctas, stream);
  }
}

}  // namespace nvfp4
