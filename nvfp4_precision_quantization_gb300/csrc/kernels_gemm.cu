// kernels_gemm.cu -- the GEMM that consumes two NVFP4 operands, on the
// fifth-generation tensor cores (tcgen05, sm_103a).
//
// What it computes ("NVFP4: enable row-scaled transpose quantization for
// backward", TransformerEngine PR #3206, sequence diagram): the fprop GEMM scales
// its output by the activation's per-row amax and the weight's amax, the wgrad
// GEMM by the outer product of both operands' per-line amax.  As a definition:
//   D[i][j] = sum_k value_A(i,k) * value_B(j,k),
//   value = code * decode(scale) * amax / (bound * 6)
// with both operands K-major (a rowwise output, or a columnwise output when the
// operand is the transpose).  The block part code * decode(scale) is exact in the
// tensor core's block-scaled MMA (kind::mxf4nvf4, one E4M3 scale per 16 values),
// which accumulates in FP32 in TMEM; the per-line factors alpha_i = amax_A[i] *
// fl(1/F_A) and beta_j = amax_B[j] * fl(1/F_B) are applied in the epilogue as
// D = fl(fl(acc * alpha_i) * beta_j) -- the bilateral post-scale, fused, so the
// accumulator never goes to HBM.
//
// Structure (persistent: one CTA per SM walks 128 x 256 output tiles, tile c,
// c + gridDim.x, ..., groups of 32 M tiles side by side so their A tiles stay in L2):
//   warp 0    producer: TMA loads of the A and B code tiles (128 B of K per row,
//             128B swizzle) and 1D bulk copies of their scales, into a 3-stage
//             shared-memory ring (72 KB a stage) guarded by mbarriers, running on
//             across tile boundaries;
//   warp 1    allocates TMEM (512 columns) and, from one thread, copies each
//             stage's scales to TMEM (tcgen05.cp) and issues the MMAs (M = 128,
//             N = 256, K = 64, four per stage), releasing each stage with
//             tcgen05.commit and the finished accumulator with one more;
//   warps 2-9 epilogue, two per TMEM lane quarter (128 columns each): before the
//             accumulator is ready, load alpha_i and stage the 128 beta_j in shared
//             memory; then copy the accumulator to registers (tcgen05.ld), hand
//             TMEM back to the MMA warp at once (the next tile's MMAs overlap the
//             rest), apply alpha_i * beta_j, convert and store D in whole 32-byte
//             sectors.
// With an epilogue (EPI: bias, activation, residual, the pre-activation kept) the same
// warps finish the tile in blocks of 32 x 32 (epilogue_block32), the residual's lines asked
// for while the MMAs run.  Measured (bias, GELU): 16384 x 28672 x 8192 1.89 ms, 1.97 with z
// kept, 3.9 PFLOP/s, 2.03 with a residual, against 1.87 ms for the product alone; 8192 x 8192
// x 2048 134 us, 149 with z, 145 with a residual, 171 with both, 96 for the product alone: with
// few K tiles the epilogue's loads and stores show.
// Scales reach the kernel in the layout their TMEM copies want (see SfLayout): a
// pre-pass (k_sf_layout) rewrites the compact [lines][k/16] scales of both operands
// into the caller's workspace.
//
// Every wait is bounded (about 2 s): on a timeout the kernel records
// NVFP4_DEVICE_TIMEOUT, stops issuing work, waits (bounded) for what it already
// issued, writes no output, frees its TMEM and returns.
#include <cuda_bf16.h>

#include <algorithm>

#include "activation.cuh"
#include "device_common.cuh"
#include "internal.h"
#include "row_io.cuh"
#include "tcgen05.cuh"

namespace nvfp4 {
namespace {

constexpr int kBM = 128;                   // tile rows of A = MMA M
constexpr int kBN = 256;                   // tile rows of B = output columns per tile = MMA N
// K bytes per stage and row: 256 E2M1 values.  (64 -- six stages of 36 KB with the
// 64B swizzle -- is correct too but measured 17 % slower.)
constexpr int kBKBytes = 128;
constexpr int kUmmaKBytes = 32;            // K = 64 values per MMA
constexpr int kKSteps = kBKBytes / kUmmaKBytes;  // MMAs per stage
constexpr int kTileScales = kBKBytes / 8;        // scales per line and K tile
// the operand tiles' shared-memory swizzle: one 8-row atom of kBKBytes-byte rows
constexpr int kSwizzleMode = kBKBytes == 128 ? 2 : 4;  // descriptor code: 128B / 64B
static_assert(kBKBytes == 128 || kBKBytes == 64, "K tile of 128 or 64 bytes per row");
constexpr int kABytes = kBM * kBKBytes;    // 16 KB
constexpr int kBBytes = kBN * kBKBytes;    // 32 KB
constexpr int kEpilogueWarps = 8;                    // two per TMEM lane quarter
constexpr int kEpiCols = kBN / 2;                     // accumulator columns per epilogue warp
constexpr int kThreads = 64 + 32 * kEpilogueWarps;    // producer, MMA, epilogue
constexpr uint32_t kTmemCols = 512;
constexpr int kSfCol0 = kBN;                          // scale columns follow the accumulator
constexpr int kMetaBytes = 1024;                      // barriers, TMEM address, error flag
constexpr int kSmemEnds = 512;                        // group ends staged in shared memory
constexpr int kBetaBytes = kEpilogueWarps * kEpiCols * 4;  // per-warp column factors

// Where the tensor core reads the scales of a block-scaled MMA with M = 128 and
// scale_vec::4X (one 32-bit TMEM word = the four scales of a line for the MMA's
// K = 64; base columns on multiples of 4): A's line l from its accumulator lane l
// at column base + l / 32; B's line n (N = 256) by each lane quarter q of the tensor
// core from its own lanes, lane 32q + n % 32, at column base + n / 32 -- B's scales
// must be present in all four quarters.  They get there by tcgen05.cp .128x256b
// (lane l <- a 32-byte row of shared memory, 8 columns): one copy holds two K steps
// of A (row l: the words of K steps 2c and 2c + 1 at bytes 4q and 16 + 4q, q = l /
// 32, zero elsewhere) or one K step of all 256 lines of B (row l: line 32c + l % 32
// at bytes 4c).  Per K tile of 256: 2 + 4 copies, 8 + 16 KB of shared memory, 16 +
// 32 TMEM columns (A's K step ks at base + 4ks, B's at base + 8ks).
struct SfLayout {
  static constexpr int kStages = kBKBytes == 128 ? 3 : 6;
  static constexpr int kSfaBytes = kKSteps / 2 * 4096;
  static constexpr int kSfbBytes = kKSteps * 4096;
  static constexpr int kSfaCols = 4 * kKSteps, kSfbCols = 8 * kKSteps;
};
template <class SF>
struct GemmGeom {
  static constexpr int kStageBytes = kABytes + kBBytes + SF::kSfaBytes + SF::kSfbBytes;
  static constexpr int kSfColsPerStage = SF::kSfaCols + SF::kSfbCols;
  static constexpr int kSmemBytes = SF::kStages * kStageBytes + kMetaBytes +
                                    kSmemEnds * 8 /* group ends */ + kBetaBytes +
                                    1024 /* alignment */;
  static_assert(kSfCol0 + SF::kStages * kSfColsPerStage <= (int)kTmemCols, "TMEM columns");
  static_assert(kStageBytes % 1024 == 0, "stages stay 1024-byte aligned for the 128B swizzle");
  static_assert(kSmemBytes <= 232448, "shared memory");
};


// Shared-memory matrix descriptor of a K-major operand tile with kBKBytes-byte rows
// in the matching swizzle: 8-row groups 8 * kBKBytes bytes apart (stride byte
// offset), the leading byte offset unused for this layout, bits 46-48 = 0b001.
__device__ __forceinline__ uint64_t desc_swz(uint32_t saddr) {
  return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)1 << 16) |
         ((uint64_t)(8 * kBKBytes >> 4) << 32) | ((uint64_t)1 << 46) |
         ((uint64_t)kSwizzleMode << 61);
}
// ---------------------------------------------------------------- scale pre-pass

// Scale pre-pass.  Compact scales [rows][k16] -> [n_blk][k_tiles][copies][4096] for
// blocks of 128 * P lines (P = 1: A, two copies per K tile; P = 2: B, four).  In
// copy c, lane l owns a 32-byte row of eight 4-byte words (the four scales of one
// line and K step each, zero where unused):
//   A (P = 1): word 4u + q (q = l / 32) of row l = line blk * 128 + l, K step 2c + u;
//   B (P = 2): word cc of row l = line blk * 256 + 32 cc + l % 32, K step c.
// Stored as one tcgen05.cp .128x256b reads it: 16-byte half u at 2048 u, row l at
// 16 l.  One CTA per (block, K tile): it stages the block's 16 scales per line of
// that K tile in shared memory (16-byte loads where the rows allow), then writes
// the block's copies as coalesced 16-byte stores, one 16-byte row half per thread.
__global__ void __launch_bounds__(256) k_sf_layout(const uint8_t* __restrict__ sc, int64_t rows,
                                                  int64_t k16, int64_t k_tiles, int P,
                                                  uint8_t* __restrict__ out) {
  __shared__ uint32_t cw[256 * kKSteps];  // cw[kKSteps * line + ks]: the line's K step ks
  const int L = 128 * P;
  const int copies = P == 1 ? kKSteps / 2 : kKSteps;
  const int64_t kt = blockIdx.x % k_tiles, blk = blockIdx.x / k_tiles;
  const int64_t s0 = kt * kTileScales;
  const bool vec = k16 % kTileScales == 0 && (reinterpret_cast<uintptr_t>(sc) & 15) == 0;
  const bool pairs = (k16 & 1) == 0 && (reinterpret_cast<uintptr_t>(sc) & 1) == 0;
  for (int i = threadIdx.x; i < L; i += blockDim.x) {
    const int64_t line = blk * L + i;
    uint32_t w[kKSteps];
#pragma unroll
    for (int j = 0; j < kKSteps; ++j) w[j] = 0;
    if (line < rows) {
      const uint8_t* p = sc + line * k16 + s0;
      if (vec) {
#pragma unroll
        for (int j = 0; j < kKSteps; ++j) w[j] = __ldg(reinterpret_cast<const uint32_t*>(p) + j);
      } else if (pairs) {
#pragma unroll
        for (int j = 0; j < kTileScales; j += 2)
          if (s0 + j < k16)
            w[j >> 2] |= (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(p + j)) << (8 * (j & 3));
      } else {
        for (int j = 0; j < kTileScales && s0 + j < k16; ++j)
          w[j >> 2] |= (uint32_t)p[j] << (8 * (j & 3));
      }
    }
#pragma unroll
    for (int j = 0; j < kKSteps; ++j) cw[kKSteps * i + j] = w[j];
  }
  __syncthreads();
  uint4* dst = reinterpret_cast<uint4*>(out + blockIdx.x * (int64_t)copies * 4096);
  for (int v = threadIdx.x; v < copies * 256; v += blockDim.x) {
    const int c = v >> 8, u = (v >> 7) & 1, l = v & 127;  // copy, half, row
    uint32_t w[4];
    if (P == 1) {  // line l, K step 2c + u, at word l / 32
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = j == (l >> 5) ? cw[kKSteps * l + 2 * c + u] : 0u;
    } else {  // words 4u .. 4u + 3: lines 32 (4u + j) + l % 32, K step c
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = cw[kKSteps * (32 * (4 * u + j) + (l & 31)) + c];
    }
    dst[u * 128 + l + c * 256] = make_uint4(w[0], w[1], w[2], w[3]);
  }
}

// ---------------------------------------------------------------- the GEMM

struct GemmParams {
  const uint8_t* sfa;  // A's scales in the kernel's layout
  const uint8_t* sfb;
  const float* a_amax;
  const float* b_amax;
  int a_amax_stride;  // 1 (per line) or 0 (per tensor)
  int b_amax_stride;
  float a_finv, b_finv;  // fl(1 / (bound * 6)) of each operand
  int M, N;
  int k_tiles;  // ceil(K / 256)
  int tiles_m, tiles_n;
  void* d;
  bool d_bf16;
  uint32_t idesc;
  int* status;
  // grouped (per-expert) GEMM: rows of A in groups ending at group_ends (multiples of
  // 128), group g multiplying rows g * b_group_rows .. of B; NULL for one GEMM
  const int64_t* group_ends;
  int num_groups;
  int b_group_rows;         // N in the grouped GEMM, 0 otherwise
  int b_amax_group_stride;  // where group g's amax starts in b_amax (N, 1 or 0)
  // K-grouped (the per-expert wgrad GEMM): group_ends cut K (tokens, multiples of 256)
  // and group g writes its own [M][N] block of d, d + g * M * N
  bool k_grouped;
  int64_t group_total;      // what the last group end must equal (rows of A, or K)
  int a_amax_group_stride;  // where group g's amax starts in a_amax (K-grouped: M, 1)
  Epilogue epi;             // k_gemm_nvf4<SF, true> only (no groups)
};

// One output tile of this CTA's walk: its group, tile coordinates and K tiles.
struct TileJob {
  int g, tm, tn, kt0, kt1;
};

// The group of the A tile starting at row r: the first g with group_ends[g] > r
// (empty groups are skipped); 0 when the GEMM is not grouped by rows.
__device__ __forceinline__ int group_of_row(const GemmParams& p, const int64_t* ends, int64_t r) {
  if (p.group_ends == nullptr || p.k_grouped) return 0;
  int lo = 0, hi = p.num_groups - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] > r) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

constexpr int kRasterGroup = 32;  // M tiles walked together so their A tiles stay in L2

__device__ __forceinline__ void tile_coords(int idx, int tiles_m, int tiles_n, int& tm, int& tn);
__device__ __forceinline__ int group_of_row(const GemmParams& p, const int64_t* ends, int64_t r);

// ends: the group ends (a shared-memory copy when they fit)
__device__ __forceinline__ TileJob tile_job(const GemmParams& p, const int64_t* ends, int tile) {
  TileJob j;
  j.g = 0;
  j.kt0 = 0;
  j.kt1 = p.k_tiles;
  if (p.k_grouped) {
    const int per = p.tiles_m * p.tiles_n;
    j.g = tile / per;
    tile_coords(tile - j.g * per, p.tiles_m, p.tiles_n, j.tm, j.tn);
    j.kt0 = (int)((j.g ? ends[j.g - 1] : 0) / (2 * kBKBytes));
    j.kt1 = (int)(ends[j.g] / (2 * kBKBytes));
  } else {
    tile_coords(tile, p.tiles_m, p.tiles_n, j.tm, j.tn);
    if (p.group_ends != nullptr) j.g = group_of_row(p, ends, (int64_t)j.tm * kBM);
  }
  return j;
}

__device__ __forceinline__ void tile_coords(int idx, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int group = idx / (kRasterGroup * tiles_n);
  const int first_m = group * kRasterGroup;
  const int gm = min(tiles_m - first_m, kRasterGroup);
  const int rem = idx - group * kRasterGroup * tiles_n;
  tm = first_m + rem % gm;
  tn = rem / gm;
}

// 32 consecutive output columns of one row, FP32 -> D's type, in 32-byte (v8) or 16-byte
// stores.
__device__ __forceinline__ void store_run32(void* base, bool bf16, int64_t off, const float* v,
                                            bool v8) {
  const int step = bf16 ? 16 : 8;  // values of a 32-byte sector
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    uint32_t w[8];
    if (bf16) {
      if (g >= 2) break;
#pragma unroll
      for (int j = 0; j < 8; ++j)
        w[j] = bf16x2_bits(v[(16 * g + 2 * j) & 31], v[(16 * g + 2 * j + 1) & 31]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(v[8 * g + j]);
    }
    char* dst = static_cast<char*>(base) + (off + g * step) * (bf16 ? 2 : 4);
    if (v8) {
      stg_v8(dst, w);
    } else {
      *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4*>(dst + 16) = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

// v[i] of lane l <- v[l] of lane i: a 32 x 32 transposition between the lanes of a warp.
__device__ __forceinline__ void transpose32(float* v, int lane) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    const bool upper = lane & d;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if (i & d) continue;
      const float got = __shfl_xor_sync(0xffffffffu, upper ? v[i] : v[i | d], d);
      if (upper) v[i] = got;
      else v[i | d] = got;
    }
  }
}

// The epilogue of a warp's 32 rows (one per lane) x 32 columns: v, the product plus bias, is
// z, kept if asked for; then act(z) + residual, stored.  Whole, aligned runs (v16) are moved
// by each lane in its own row.  Otherwise every lane's
// accesses would start and end anywhere (an odd N measured four times slower), so the block
// is transposed and a request covers 32 neighbouring columns of a row.
struct EpilogueBlock {
  int row0, col0;  // of the block
  int rows, cols;  // of it, inside D
};
__device__ __forceinline__ void epilogue_block32(const GemmParams& p, const EpilogueBlock& b,
                                                 float* v, bool v16, bool v8, int lane) {
  const Epilogue& e = p.epi;
  if (v16) {
    const int64_t off = (int64_t)(b.row0 + lane) * p.N + b.col0;
    const bool live = lane < b.rows;
    if (e.z != nullptr && live) store_run32(e.z, p.d_bf16, off, v, v8);
    if (e.residual != nullptr && p.d_bf16) {  // in flight during the activation
      Chunk<true> r[2];
#pragma unroll
      for (int c = 0; c < 2; ++c)
        r[c].load(e.residual, off + kChunk * c, live ? kChunk : 0, v8 ? 32 : 16);
      apply_act<32>(e.act, v);
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = __fadd_rn(v[j], r[j / kChunk].get(j % kChunk));
      if (live) store_run32(p.d, true, off, v, v8);
      return;
    }
    apply_act<32>(e.act, v);
    if (e.residual != nullptr) {
#pragma unroll
      for (int c = 0; c < 32; c += kChunk) {
        float r[kChunk];
        load_vector16(e.residual, p.d_bf16, off + c, live ? kChunk : 0, v8 ? 32 : 16, r);
#pragma unroll
        for (int j = 0; j < kChunk; ++j) v[c + j] = __fadd_rn(v[c + j], r[j]);
      }
    }
    if (live) store_run32(p.d, p.d_bf16, off, v, v8);
    return;
  }
  transpose32(v, lane);  // v[i]: row row0 + i, column col0 + lane
  const bool live = lane < b.cols;
  const int64_t off = (int64_t)b.row0 * p.N + b.col0 + lane;
  auto store = [&](void* base) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      if (!live || i >= b.rows) continue;
      if (p.d_bf16)
        static_cast<__nv_bfloat16*>(base)[off + (int64_t)i * p.N] = __float2bfloat16_rn(v[i]);
      else
        static_cast<float*>(base)[off + (int64_t)i * p.N] = v[i];
    }
  };
  if (e.z != nullptr) store(e.z);
  apply_act<32>(e.act, v);
  if (e.residual != nullptr) {
#pragma unroll
    for (int g = 0; g < 32; g += 8) {
      float r[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        r[i] = 0.0f;
        if (!live || g + i >= b.rows) continue;
        const int64_t at = off + (int64_t)(g + i) * p.N;
        r[i] = p.d_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(e.residual)[at])
                        : static_cast<const float*>(e.residual)[at];
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[g + i] = __fadd_rn(v[g + i], r[i]);
    }
  }
  store(p.d);
}
// Persistent: CTA c computes tiles c, c + gridDim.x, ...  The load ring runs on
// across tile boundaries; the epilogue copies the accumulator to registers,
// hands TMEM back (acc_empty) and stores while the MMAs of the next tile run.
// EPI: with bias, activation and residual (p.epi) applied to the scaled accumulator.
template <class SF, bool EPI>
__global__ void __launch_bounds__(kThreads, 1)
    k_gemm_nvf4(const __grid_constant__ CUtensorMap map_a,
                const __grid_constant__ CUtensorMap map_b, const GemmParams p) {
  using G = GemmGeom<SF>;
  constexpr int S = SF::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S * G::kStageBytes);
  uint64_t* empty = full + S;
  uint64_t* acc_full = empty + S;
  uint64_t* acc_empty = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 1);
  int* err = reinterpret_cast<int*>(tmem_slot + 1);
  int64_t* s_ends = reinterpret_cast<int64_t*>(smem + S * G::kStageBytes + kMetaBytes);
  float* s_beta = reinterpret_cast<float*>(s_ends + kSmemEnds);
  // every tile looks its group up: from shared memory when the ends fit
  const int64_t* ends = p.num_groups <= kSmemEnds ? s_ends : p.group_ends;
  if (p.group_ends != nullptr && p.num_groups <= kSmemEnds)
    for (int g = threadIdx.x; g < p.num_groups; g += blockDim.x) s_ends[g] = p.group_ends[g];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int num_tiles = (p.k_grouped ? p.num_groups : 1) * p.tiles_m * p.tiles_n;

  if (p.group_ends != nullptr) {  // every thread takes part; nothing is written if invalid
    const bool ok = groups_valid(p.group_ends, p.num_groups, p.group_total) &&
                    ends_aligned(p.group_ends, p.num_groups, p.k_grouped ? 2 * kBKBytes : kBM);
    if (!ok) {
      if (threadIdx.x == 0) raise_status(p.status, kStatusBadGroups);
      return;
    }
  }

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, kEpilogueWarps);
    *err = 0;
    fence_mbar_init();
    prefetch_tmap(&map_a);
    prefetch_tmap(&map_b);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0 && lane == 0) {
    // ---------------- producer
    const uint64_t pol_a = policy_evict_last();
    const uint64_t pol_b = policy_evict_normal();
    uint32_t it = 0;  // K tiles issued, over all tiles of this CTA
    bool ok = true;
    for (int tile = blockIdx.x; ok && tile < num_tiles; tile += gridDim.x) {
      const TileJob job = tile_job(p, ends, tile);
      const int tm = job.tm, tn = job.tn;
      const int b_tile0 = job.g * (p.b_group_rows / kBN);  // the expert's rows of B
      for (int kt = job.kt0; kt < job.kt1; ++kt, ++it) {
        const uint32_t s = it % S;
        if (it >= (uint32_t)S && !mbar_wait_bounded(&empty[s], ((it / S) - 1) & 1)) {
          *err = 1;
          ok = false;
          break;
        }
        if (*(volatile int*)err) {
          ok = false;
          break;
        }
        uint8_t* st = smem + s * G::kStageBytes;
        uint8_t* st_sf = st + kABytes + kBBytes;
        mbar_expect_tx(&full[s], G::kStageBytes);
        const int bt = b_tile0 + tn;  // B's 256-row tile (of its group)
        tma_load_2d(st, &map_a, &full[s], kt * kBKBytes, tm * kBM, pol_a);
        tma_load_2d(st + kABytes, &map_b, &full[s], kt * kBKBytes, bt * kBN, pol_b);
        bulk_load(st_sf, p.sfa + ((int64_t)tm * p.k_tiles + kt) * SF::kSfaBytes, SF::kSfaBytes,
                  &full[s], pol_a);
        bulk_load(st_sf + SF::kSfaBytes, p.sfb + ((int64_t)bt * p.k_tiles + kt) * SF::kSfbBytes,
                  SF::kSfbBytes, &full[s], pol_b);
      }
    }
    // drain: every copy issued must have landed before the CTA may exit
    for (uint32_t j = it > (uint32_t)S ? it - S : 0; j < it; ++j)
      if (!mbar_wait_bounded(&full[j % S], (j / S) & 1)) *err = 1;
  } else if (warp == 1 && lane == 0) {
    // ---------------- MMA issuer: per K tile, the stage's scales to TMEM, then
    // the four MMAs (K = 64 each) that read them
    auto copy_scales = [&](uint32_t j) {
      const uint32_t s = j % S;
      const uint32_t st_sfa = smem_addr(smem + s * G::kStageBytes) + kABytes + kBBytes;
      const uint32_t st_sfb = st_sfa + SF::kSfaBytes;
      const uint32_t sfa_col = tmem + kSfCol0 + s * G::kSfColsPerStage;
      const uint32_t sfb_col = sfa_col + SF::kSfaCols;
      // 128 rows x 32 bytes per copy: 16-byte halves 2048 bytes apart, rows 16 apart
#pragma unroll
      for (int c = 0; c < kKSteps / 2; ++c)
        tc_cp_128x256b(sfa_col + 8 * c, desc_plain(st_sfa + c * 4096, 2048, 128));
#pragma unroll
      for (int ks = 0; ks < kKSteps; ++ks)
        tc_cp_128x256b(sfb_col + 8 * ks, desc_plain(st_sfb + ks * 4096, 2048, 128));
    };
    uint32_t it = 0, t = 0;
    bool ok = true;
    for (int tile = blockIdx.x; ok && tile < num_tiles; tile += gridDim.x, ++t) {
      // the epilogue of the previous tile has copied the accumulator out
      if (t > 0 && !mbar_wait_bounded(acc_empty, (t - 1) & 1)) {
        *err = 1;
        break;
      }
      tc_fence_after();
      const TileJob job = tile_job(p, ends, tile);
      for (int kt = job.kt0; kt < job.kt1; ++kt, ++it) {
        const uint32_t s = it % S;
        if (!mbar_wait_bounded(&full[s], (it / S) & 1)) {
          *err = 1;
          ok = false;
          break;
        }
        if (*(volatile int*)err) {
          ok = false;
          break;
        }
        tc_fence_after();
        copy_scales(it);
        const uint32_t st = smem_addr(smem + s * G::kStageBytes);
        const uint32_t sfa_col = tmem + kSfCol0 + s * G::kSfColsPerStage;
        const uint32_t sfb_col = sfa_col + SF::kSfaCols;
#pragma unroll
        for (int ks = 0; ks < kKSteps; ++ks)
          tc_mma_nvf4(tmem, desc_swz(st + ks * kUmmaKBytes),
                      desc_swz(st + kABytes + ks * kUmmaKBytes), p.idesc, sfa_col + 4 * ks,
                      sfb_col + 8 * ks, (kt != job.kt0) || ks != 0);
        tc_commit(&empty[s]);
      }
      // the accumulator of this tile is complete (or abandoned) once all issued MMAs are
      tc_commit(acc_full);
    }
    // everything issued must be done before TMEM is freed
    if (t > 0 && !mbar_wait_bounded(acc_full, (t - 1) & 1)) *err = 1;
  } else if (warp >= 2) {
    // ---------------- epilogue: lane quarter q (rows 32q ..), column half `half`
    const int q = warp & 3;
    const int half = (warp - 2) >> 2;
    const bool b_lines = p.b_amax_stride != 0;  // one amax per line of B
    uint32_t t = 0;
    float* beta = s_beta + (warp - 2) * kEpiCols;  // this warp's column factors
    // and its bias, where a grouped GEMM keeps its group ends
    float* bias = reinterpret_cast<float*>(s_ends) + (warp - 2) * kEpiCols;
    for (int tile = blockIdx.x; tile < num_tiles; tile += gridDim.x, ++t) {
      const TileJob job = tile_job(p, ends, tile);
      const int tm = job.tm, tn = job.tn;
      const int row = tm * kBM + q * 32 + lane;
      const int col_base = tn * kBN + half * kEpiCols;
      const bool live = row < p.M && col_base < p.N;
      // Before the accumulator is ready: alpha = fl(amax_a[row] * fl(1/F_a)) and this
      // warp's 128 column factors beta = fl(amax_b[col] * fl(1/F_b)), lane l computing
      // columns 4l .. 4l+3 into shared memory, so that no global load waits behind
      // the accumulator.
      const float alpha =
          live ? __fmul_rn(p.a_amax[(int64_t)job.g * p.a_amax_group_stride +
                                    (int64_t)row * p.a_amax_stride],
                           p.a_finv)
               : 0.f;
      {
        const float* b_amax = p.b_amax + (int64_t)job.g * p.b_amax_group_stride;
        const int c4 = col_base + 4 * lane;
        float b4[4];
        // 16-byte loads only where this group's amax row is 16-byte aligned
        if (b_lines && (reinterpret_cast<uintptr_t>(b_amax) & 15) == 0 && c4 + 4 <= p.N) {
          const float4 t4 = __ldg(reinterpret_cast<const float4*>(b_amax + c4));
          b4[0] = t4.x, b4[1] = t4.y, b4[2] = t4.z, b4[3] = t4.w;
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            b4[j] = __ldg(b_amax + (int64_t)max(0, min(c4 + j, p.N - 1)) * p.b_amax_stride);
        }
        __syncwarp();  // every lane has read the previous tile's factors
        sts_v4(beta + 4 * lane, __float_as_uint(__fmul_rn(b4[0], p.b_finv)),
               __float_as_uint(__fmul_rn(b4[1], p.b_finv)),
               __float_as_uint(__fmul_rn(b4[2], p.b_finv)),
               __float_as_uint(__fmul_rn(b4[3], p.b_finv)));
        if constexpr (EPI) {  // and its bias
          float c[4];
#pragma unroll
          for (int j = 0; j < 4; ++j)
            c[j] = p.epi.bias_at(c4 + j < p.N ? c4 + j : -1);
          sts_v4(bias + 4 * lane, __float_as_uint(c[0]), __float_as_uint(c[1]),
                 __float_as_uint(c[2]), __float_as_uint(c[3]));
        }
        __syncwarp();
      }
      if constexpr (EPI) {
        // the warp's part of the residual into L2 while the MMAs run: 128-byte lines, each
        // lane those of its row
        if (live && p.epi.residual != nullptr) {
          const int esize = p.d_bf16 ? 2 : 4;
          const char* from = static_cast<const char*>(p.epi.residual) +
                             ((int64_t)row * p.N + col_base) * esize;
          const int bytes = min(kEpiCols, p.N - col_base) * esize;
          for (int b = 0; b < bytes; b += 128)
            asm volatile("prefetch.global.L2 [%0];" ::"l"(from + b));
        }
      }
      const bool ready = mbar_wait_bounded(acc_full, t & 1);
      if (!ready) *err = 1;
      tc_fence_after();
      uint32_t v[kEpiCols];
#pragma unroll
      for (int c = 0; c < kEpiCols / 32; ++c)
        tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + half * kEpiCols + c * 32, v + c * 32);
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acc_empty);  // TMEM may take the next tile's MMAs
      // the warp leaves together: what follows (shuffles, the next tile's TMEM loads) takes
      // every lane, and each lane's wait gives up by its own clock
      if (__any_sync(0xffffffffu, !ready || *(volatile int*)err)) break;
      if (job.kt1 == job.kt0) {  // an empty K range (an empty group): the sum is 0
#pragma unroll
        for (int i = 0; i < kEpiCols; ++i) v[i] = 0u;
      }
      if constexpr (EPI) {
        // the warp's rows and columns inside D; every lane takes part
        const int rows = min(32, p.M - (tm * kBM + q * 32));
        const int cols = min(kEpiCols, p.N - col_base);
        if (rows <= 0 || cols <= 0) continue;
        const int esize = p.d_bf16 ? 2 : 4;
        uintptr_t align = reinterpret_cast<uintptr_t>(p.d) | (uintptr_t)p.N * esize;
        if (p.epi.residual) align |= reinterpret_cast<uintptr_t>(p.epi.residual);
        if (p.epi.z) align |= reinterpret_cast<uintptr_t>(p.epi.z);
        const bool v16 = cols == kEpiCols && (align & 15) == 0, v8 = (align & 31) == 0;
#pragma unroll
        for (int c = 0; c < kEpiCols / 32; ++c) {
          if (c * 32 >= cols) break;
          float f[32];
          // d = fl(fl(acc * alpha) * beta) + bias
#pragma unroll
          for (int j4 = 0; j4 < 8; ++j4) {
            const float4 b4 = *reinterpret_cast<const float4*>(beta + c * 32 + 4 * j4);
            const float4 a4 = *reinterpret_cast<const float4*>(bias + c * 32 + 4 * j4);
            const float bj[4] = {b4.x, b4.y, b4.z, b4.w}, aj[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              f[4 * j4 + j] = __fadd_rn(
                  __fmul_rn(__fmul_rn(__uint_as_float(v[c * 32 + 4 * j4 + j]), alpha), bj[j]),
                  aj[j]);
          }
          epilogue_block32(p, {tm * kBM + q * 32, col_base + c * 32, rows, min(32, cols - c * 32)},
                           f, v16, v8, lane);
        }
        continue;
      }
      if (!live) continue;
      const int nvalid = min(kEpiCols, p.N - col_base);
      const int64_t off = (p.k_grouped ? (int64_t)job.g * p.M * p.N : 0) +
                          (int64_t)row * p.N + col_base;
      // whole 32-byte sectors per store where the row's run is 32-byte aligned,
      // else 16-byte stores, else (ragged N or odd alignment) element stores
      const uintptr_t d_addr = reinterpret_cast<uintptr_t>(p.d) + off * (p.d_bf16 ? 2 : 4);
      const bool vec = nvalid == kEpiCols && (d_addr & 15) == 0;
      const bool vec32 = vec && (d_addr & 31) == 0;
#pragma unroll
      for (int c = 0; c < kEpiCols / 32; ++c) {
        uint32_t* vc = v + c * 32;
        // d = fl(fl(acc * alpha) * beta)
#pragma unroll
        for (int j4 = 0; j4 < 8; ++j4) {
          const float4 b4 = *reinterpret_cast<const float4*>(beta + c * 32 + 4 * j4);
          const float bj[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
          for (int j = 0; j < 4; ++j)
            vc[4 * j4 + j] =
                __float_as_uint(__fmul_rn(__fmul_rn(__uint_as_float(vc[4 * j4 + j]), alpha), bj[j]));
        }
        if (p.d_bf16) {
          uint16_t* dst = static_cast<uint16_t*>(p.d) + off + c * 32;
          uint32_t w[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            __nv_bfloat162 h2 = __floats2bfloat162_rn(__uint_as_float(vc[2 * j]),
                                                      __uint_as_float(vc[2 * j + 1]));
            w[j] = *reinterpret_cast<uint32_t*>(&h2);
          }
          if (vec32) {
            stg_v8(dst, w);
            stg_v8(dst + 16, w + 8);
          } else if (vec) {
#pragma unroll
            for (int g = 0; g < 4; ++g)
              *reinterpret_cast<uint4*>(dst + 8 * g) =
                  make_uint4(w[4 * g], w[4 * g + 1], w[4 * g + 2], w[4 * g + 3]);
          } else {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (c * 32 + j < nvalid) dst[j] = (uint16_t)(w[j >> 1] >> (16 * (j & 1)));
          }
        } else {
          uint32_t* dst = static_cast<uint32_t*>(p.d) + off + c * 32;
#pragma unroll
          for (int g = 0; g < 8; ++g) {
            if (vec32) {
              if ((g & 1) == 0) stg_v8(dst + 4 * g, vc + 4 * g);
            } else if (vec) {
              *reinterpret_cast<uint4*>(dst + 4 * g) =
                  make_uint4(vc[4 * g], vc[4 * g + 1], vc[4 * g + 2], vc[4 * g + 3]);
            } else {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (c * 32 + 4 * g + j < nvalid) dst[4 * g + j] = vc[4 * g + j];
            }
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *(volatile int*)err) raise_status(p.status, kStatusTimeout);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// d = act(bias) + residual: the epilogue of an empty sum (k == 0), two elements at a time
// because the activations' one form is of pairs.
__global__ void __launch_bounds__(256) k_epilogue_only(const Epilogue e, void* d, bool bf16,
                                                       int64_t m, int n) {
  const int64_t total = m * n;
  auto put = [&](void* base, int64_t i, float v) {
    if (bf16) static_cast<__nv_bfloat16*>(base)[i] = __float2bfloat16_rn(v);
    else static_cast<float*>(base)[i] = v;
  };
  for (int64_t i = 2 * ((int64_t)blockIdx.x * 256 + threadIdx.x); i < total;
       i += 2 * (int64_t)gridDim.x * 256) {
    const int count = i + 1 < total ? 2 : 1;
    float v[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) v[j] = j < count ? e.bias_at((int)((i + j) % n)) : 0.0f;
    if (e.z != nullptr)
      for (int j = 0; j < count; ++j) put(e.z, i + j, v[j]);
    apply_act<2>(e.act, v);
    for (int j = 0; j < count; ++j) {
      float r = 0.0f;
      if (e.residual != nullptr)
        r = bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(e.residual)[i + j])
                 : static_cast<const float*>(e.residual)[i + j];
      put(d, i + j, e.residual != nullptr ? __fadd_rn(v[j], r) : v[j]);
    }
  }
}

}  // namespace

cudaError_t launch_epilogue_only(const Epilogue& e, void* d, bool bf16, int64_t m, int64_t n,
                                 const DeviceInfo& dev, cudaStream_t stream) {
  const int64_t grid = std::min<int64_t>((m * n + 511) / 512, 8LL * dev.num_sms);
  k_epilogue_only<<<(unsigned)grid, 256, 0, stream>>>(e, d, bf16, m, (int)n);
  return cudaGetLastError();
}

GemmLayout gemm_layout(int64_t M, int64_t N, int64_t K, int64_t b_lines) {
  GemmLayout L;
  L.k_tiles = ceil_div(K, 2 * kBKBytes);
  L.tiles_m = ceil_div(M, kBM);
  L.tiles_n = ceil_div(N, kBN);
  L.sfa_bytes = L.tiles_m * L.k_tiles * SfLayout::kSfaBytes;
  L.sfb_bytes = ceil_div(b_lines, kBN) * L.k_tiles * SfLayout::kSfbBytes;
  L.sfb_offset = (L.sfa_bytes + 255) / 256 * 256;
  L.workspace_bytes = L.sfb_offset + L.sfb_bytes;
  return L;
}

template <class SF, bool EPI>
static cudaError_t launch_gemm_t(const GemmArgs& a, const GemmLayout& L, const DeviceInfo& dev,
                                 cudaStream_t stream) {
  using G = GemmGeom<SF>;
  uint8_t* sfa = a.workspace;
  uint8_t* sfb = a.workspace + L.sfb_offset;
  k_sf_layout<<<(unsigned)(L.tiles_m * L.k_tiles), 256, 0, stream>>>(a.a_scales, a.M, a.K / 16,
                                                                     L.k_tiles, 1, sfa);
  const int64_t b_lines = a.group_ends && !a.k_grouped ? (int64_t)a.num_groups * a.N : a.N;
  k_sf_layout<<<(unsigned)(ceil_div(b_lines, kBN) * L.k_tiles), 256, 0, stream>>>(
      a.b_scales, b_lines, a.K / 16, L.k_tiles, 2, sfb);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;

  CUtensorMap map_a, map_b;
  if (!make_operand_map(&map_a, a.a_codes, a.M, a.K / 2, kBKBytes, kBM) ||
      !make_operand_map(&map_b, a.b_codes, b_lines, a.K / 2, kBKBytes, kBN))
    return cudaErrorInvalidValue;

  static bool attr_set[64] = {};
  if (dev.device < 64 && !attr_set[dev.device]) {
    e = cudaFuncSetAttribute(k_gemm_nvf4<SF, EPI>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             G::kSmemBytes);
    if (e != cudaSuccess) return e;
    attr_set[dev.device] = true;
  }
  GemmParams p;
  p.sfa = sfa;
  p.sfb = sfb;
  p.a_amax = a.a_amax;
  p.b_amax = a.b_amax;
  p.a_amax_stride = a.a_row_scaled ? 1 : 0;
  p.b_amax_stride = a.b_row_scaled ? 1 : 0;
  p.a_finv = 1.0f / (a.a_bound * 6.0f);
  p.b_finv = 1.0f / (a.b_bound * 6.0f);
  p.M = (int)a.M;
  p.N = (int)a.N;
  p.k_tiles = (int)L.k_tiles;
  p.tiles_m = (int)L.tiles_m;
  p.tiles_n = (int)L.tiles_n;
  p.d = a.d;
  p.d_bf16 = a.d_bf16;
  p.idesc = make_idesc_nvf4(kBM, kBN);
  p.status = dev.status;
  p.group_ends = a.group_ends;
  p.num_groups = a.group_ends ? a.num_groups : 0;
  p.k_grouped = a.group_ends != nullptr && a.k_grouped;
  p.b_group_rows = a.group_ends && !a.k_grouped ? (int)a.N : 0;
  p.b_amax_group_stride = a.group_ends ? (a.b_row_scaled ? (int)a.N : 1) : 0;
  p.a_amax_group_stride = p.k_grouped ? (a.a_row_scaled ? (int)a.M : 1) : 0;
  p.group_total = p.k_grouped ? a.K : a.M;
  const int64_t tiles = (a.group_ends && a.k_grouped ? a.num_groups : 1) * L.tiles_m * L.tiles_n;
  const int grid = (int)std::min<int64_t>(tiles, dev.num_sms);
  if constexpr (EPI) p.epi = *a.epilogue;
  k_gemm_nvf4<SF, EPI><<<grid, kThreads, G::kSmemBytes, stream>>>(map_a, map_b, p);
  return cudaGetLastError();
}

cudaError_t launch_gemm(const GemmArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  const GemmLayout L = gemm_layout(
      a.M, a.N, a.K, a.group_ends && !a.k_grouped ? (int64_t)a.num_groups * a.N : a.N);
  return a.epilogue != nullptr ? launch_gemm_t<SfLayout, true>(a, L, dev, stream)
                               : launch_gemm_t<SfLayout, false>(a, L, dev, stream);
}

}  // namespace nvfp4
