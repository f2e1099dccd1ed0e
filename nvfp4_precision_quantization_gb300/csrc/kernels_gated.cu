// kernels_gated.cu -- the gated product of two NVFP4 operands for many rows of A:
//   D [M][N] = act(A Bg^T + bg) (A Bu^T + bu),  B's 2N lines the gate's and then the up's,
// with the two projections, the activation and their product in one kernel, on pairs of SMs.
//
// Bound by the tensor cores and by what feeds them.  A pair of CTAs (a cluster of two) computes
// tiles of 256 rows x 128 columns of D: an MMA of M = 256 over both SMs, whose N = 256 lines of B
// are 128 of the gate and the 128 of the same columns of the up projection, so that a thread
// of the epilogue finds both factors of its outputs in its own accumulator row.  Of each K tile
// (256 values) a CTA loads its own 128 rows of A and one half of B's lines: 38 KB for 128 x 256
// sums, where an SM on its own would take 54.
//
// Structure (persistent: pair c walks the tiles c, c + pairs, ..., groups of 16 M tiles side by
// side so their A tiles stay in L2):
//   warp 0     producer, in both CTAs: loads of codes (TMA, 128 B of K per row, 128B swizzle),
//              which complete on the leader's (rank 0's) barriers, and of scales, on the CTA's
//              own, into a ring of kStages stages;
//   warp 1     TMEM; in the leader, one thread issues the MMAs, then releases the stage and,
//              after a tile, the accumulators, in both CTAs (tcgen05.commit, multicast);
//   warps 4-7  scales, in both CTAs, one per TMEM lane quarter: from the stage through
//              registers into tensor memory;
//   warps 8-15 epilogue, in both CTAs, two per TMEM lane quarter (64 columns of D each):
//              accumulators to registers, TMEM handed back to the leader, then bias,
//              activation, product, maxima and stores while the next tile's MMAs run.
// A pre-pass (k_gated_scales) rewrites the compact scales into 512-byte pieces of 128 lines x 4
// scales, line l at byte (l % 32) 16 + (l / 32) 4: what lane l % 32 of every lane quarter holds for
// a K step, and clears the maxima.
//
// The scales go through registers because a tcgen05.cp takes about 50 cycles of the MMAs' own
// in-order pipe whatever it moves, and a K tile would need twelve (six of the largest form): 8192 x
// 14336 x 8192 takes 1122 us so, 646 this way, 649 with the copies left out.  Measured, SILU: 16384 x
// 14336 x 8192 with [g | u] and the maxima kept 1390 us in bursts of tens of calls, 5.5 PFLOP/s, and 1500
// once they follow one another for more than a second (at 1.35 kW the SM clock goes from 2070 to 1790
// MHz); 8192 rows without them 646 us, 6.0 PFLOP/s, of which 60 us are the epilogue's.  What is left is
// the pair's walk through the ring: a K tile takes 0.42 us, 0.37 with one MMA instead of four, 0.36
// without the scales' stores; half of B's bytes, four stages instead of five or a second producer
// change nothing.
//
// Every wait is bounded, as in kernels_gemm.cu; the CTAs of a pair meet before either leaves.
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "activation.cuh"
#include "gemm_tile.cuh"
#include "internal.h"
#include "tcgen05.cuh"

namespace nvfp4 {
namespace {

constexpr int kRows = 128;                 // rows of A per CTA
constexpr int kCols = 128;                 // columns of D per tile
constexpr int kKBytes = 128;               // of a line per K tile: 256 values
constexpr int kKScales = kKBytes / 8;
constexpr int kKSteps = kKBytes / 32;      // MMAs per K tile, 64 values each
constexpr int kStages = 5;
constexpr int kABytes = kRows * kKBytes;
constexpr int kBBytes = kCols * kKBytes;   // this CTA's half of B's lines
constexpr int kPiece = 512;                // scales of 128 lines and one K step
constexpr int kSfaBytes = kKSteps * kPiece;
constexpr int kSfbBytes = 2 * kSfaBytes;   // of all 256 lines
constexpr int kStageBytes_ = kABytes + kBBytes + kSfaBytes + kSfbBytes;
constexpr int kScaleWarp0 = 4, kScaleWarps = 4;  // one per TMEM lane quarter
constexpr int kEpilogueWarp0 = 8, kEpilogueWarps = 8;
constexpr int kWarpCols = kCols / 2;       // columns of D per epilogue warp
constexpr int kThreads = 32 * (kEpilogueWarp0 + kEpilogueWarps);
// Registers by warpgroup (producer and MMA, scales, epilogue twice): an epilogue thread holds 128
// accumulators, so the others give theirs up.  The shares add up to what the block is launched
// with, 128 each.
constexpr int kRegsIssue = 64, kRegsScales = 96, kRegsEpilogue = 176;
static_assert(kRegsIssue + kRegsScales + 2 * kRegsEpilogue == 4 * 65536 / kThreads, "registers");
constexpr uint32_t kTmemCols = 512;
constexpr int kSfCol0 = 2 * kCols;         // scale columns follow the accumulators
constexpr int kSfCols = 12 * kKSteps;      // per stage: 4 of A and 8 of B per K step
constexpr int kFactorBytes = kEpilogueWarps * 4 * kWarpCols * 4;  // beta, bias of both halves
constexpr int kSmemBytes = kStages * kStageBytes_ + kFactorBytes + 512 /* barriers */ +
                           1024 /* alignment */;
static_assert(kSfCol0 + kStages * kSfCols <= (int)kTmemCols, "TMEM columns");
static_assert(kStageBytes_ % 1024 == 0, "stages stay 1024-byte aligned for the 128B swizzle");
static_assert(kSmemBytes <= 232448, "shared memory");

constexpr int kRasterGroup = 16;  // M tiles walked together so their A tiles stay in L2

struct GatedParams {
  const uint8_t* sfa;  // the pre-pass's scales
  const uint8_t* sfb;
  const float* a_amax;
  const float* b_amax;
  int a_amax_stride, b_amax_stride;  // 1 (per line) or 0 (per tensor)
  float a_finv, b_finv;              // fl(1 / (bound * 6)) of each operand
  int m, n;
  int k_tiles, tiles_m, tiles_n;
  void* d;
  bool d_bf16;
  Epilogue epi;  // bias and act
  GatedOut out;
  uint32_t idesc;
  int* status;
};

// The low bits that the rows of D and gu start with.
__host__ __device__ inline uintptr_t alignment(const GatedParams& p) {
  return reinterpret_cast<uintptr_t>(p.d) | reinterpret_cast<uintptr_t>(p.out.gu) |
         (uintptr_t)p.n * (p.d_bf16 ? 2 : 4);
}

__device__ __forceinline__ void tile_at(const GatedParams& p, int tile, int& tm, int& tn) {
  const int group = tile / (kRasterGroup * p.tiles_n), first = group * kRasterGroup;
  const int gm = min(p.tiles_m - first, kRasterGroup);
  const int rem = tile - group * kRasterGroup * p.tiles_n;
  tm = first + rem % gm;
  tn = rem / gm;
}

// ---------------------------------------------------------------- scales

struct ScaleArgs {
  const uint8_t* a;
  const uint8_t* b;
  int64_t m, n, k16;
  int k_tiles;
  int a_blocks, b_blocks;  // of 128 lines: A's; B's, gate and up by turns
  uint8_t* out;            // [a_blocks][k_tiles], then [b_blocks / 2][k_tiles][2] times kSfaBytes
  float* row_amax;         // cleared, as is col_amax
  float* col_amax;
};

// A CTA takes 128 lines and four K tiles: 64 bytes of each line to shared memory, then 16 bytes
// of the output per thread, the words of lines r, r + 32, r + 64, r + 96.
constexpr int kScaleTiles = 4;
__global__ void __launch_bounds__(256) k_gated_scales(const ScaleArgs a) {
  __shared__ uint32_t words[kRows][kScaleTiles * kKSteps + 1];
  pdl_launch_dependents();  // the product is set up meanwhile
  const int groups = (a.k_tiles + kScaleTiles - 1) / kScaleTiles;
  const int blk = blockIdx.x / groups, kt0 = blockIdx.x % groups * kScaleTiles;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.m + a.n;
       i += (int64_t)gridDim.x * 256) {
    if (i < a.m) {
      if (a.row_amax != nullptr) a.row_amax[i] = 0.0f;
    } else if (a.col_amax != nullptr) {
      a.col_amax[i - a.m] = 0.0f;
    }
  }
  // lines [first, end) of sc
  const bool is_a = blk < a.a_blocks;  // [a_blocks][k_tiles]; [b_blocks / 2][k_tiles][2]
  const int bb = blk - a.a_blocks, half = bb & 1;
  const uint8_t* sc = is_a ? a.a : a.b;
  const int64_t first = is_a ? (int64_t)blk * kRows : half * a.n + (int64_t)(bb >> 1) * kRows;
  const int64_t end = is_a ? a.m : (half + 1) * a.n;
  const int64_t s0 = (int64_t)kt0 * kKScales;
  const bool vec = a.k16 % 16 == 0 && (reinterpret_cast<uintptr_t>(sc) & 15) == 0;
  const bool pairs = a.k16 % 2 == 0 && (reinterpret_cast<uintptr_t>(sc) & 1) == 0;
  for (int i = threadIdx.x; i < kRows * kScaleTiles; i += 256) {
    const int l = i / kScaleTiles, c = i % kScaleTiles;  // 16 scales of line l
    const int64_t line = first + l, s = s0 + 16 * c;
    uint32_t w[4] = {0, 0, 0, 0};
    if (line < end && s < a.k16) {
      const uint8_t* p = sc + line * a.k16 + s;
      if (vec) {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
      } else if (pairs) {
#pragma unroll
        for (int j = 0; j < 16; j += 2)
          if (s + j < a.k16)
            w[j >> 2] |= (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(p + j)) << (8 * (j & 3));
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (s + j < a.k16) w[j >> 2] |= (uint32_t)__ldg(p + j) << (8 * (j & 3));
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) words[l][4 * c + j] = w[j];
  }
  __syncthreads();
  // a block's K tiles follow one another (A) or alternate with the other half's (B)
  const int64_t tile0 = is_a ? (int64_t)blk * a.k_tiles + kt0
                             : (int64_t)a.a_blocks * a.k_tiles +
                                   ((int64_t)(bb >> 1) * a.k_tiles + kt0) * 2 + half;
  uint4* out = reinterpret_cast<uint4*>(a.out + tile0 * kSfaBytes);
  const int steps = min(kScaleTiles, a.k_tiles - kt0) * kKSteps;
  for (int i = threadIdx.x; i < 32 * steps; i += 256) {
    const int ks = i >> 5, r = i & 31, kt = ks / kKSteps;
    out[i + (is_a ? 0 : kt * kSfaBytes / 16)] =
        make_uint4(words[r][ks], words[r + 32][ks], words[r + 64][ks], words[r + 96][ks]);
  }
}

// ---------------------------------------------------------------- epilogue

// The maxima of 32 lanes' values v[0 .. 32): lane l gets that of v[l].
__device__ __forceinline__ float lanes_max32(const float* v, int lane) {
  float t[16];
  const bool up = lane & 16;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float give = up ? v[j] : v[j + 16], keep = up ? v[j + 16] : v[j];
    t[j] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, 16));
  }
#pragma unroll
  for (int d = 8; d > 0; d >>= 1) {
    const bool upper = lane & d;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (j >= d) continue;
      const float give = upper ? t[j] : t[j + d], keep = upper ? t[j + d] : t[j];
      t[j] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, give, d));
    }
  }
  return t[0];
}

// non-negative floats are ordered like their bits, and a maximum does not depend on its order
__device__ __forceinline__ void raise(float* to, float v) {
  atomicMax(reinterpret_cast<int*>(to), __float_as_int(v));
}

// 32 consecutive output columns of one row (`cols` of them exist, a whole number of 16-byte
// units), in 32-byte (v8) or 16-byte stores.
__device__ __forceinline__ void store_cols32(void* base, bool bf16, int64_t off, const float* v,
                                             int cols, bool v8) {
  if (cols >= 32) {
    store_run32(base, bf16, off, v, v8);
    return;
  }
  if (bf16) {
#pragma unroll
    for (int j = 0; j < 32; j += 8)
      if (j < cols)
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(base) + off + j) =
            make_uint4(bf16x2_bits(v[j], v[j + 1]), bf16x2_bits(v[j + 2], v[j + 3]),
                       bf16x2_bits(v[j + 4], v[j + 5]), bf16x2_bits(v[j + 6], v[j + 7]));
  } else {
#pragma unroll
    for (int j = 0; j < 32; j += 4)
      if (j < cols)
        *reinterpret_cast<float4*>(static_cast<float*>(base) + off + j) =
            make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
  }
}

// A warp's 32 rows (one per lane) x 32 columns of D inside D (rows, cols of them): g and u are
// the projections with their bias.  ALIGNED: rows of D and gu start on 16 bytes, and each lane
// moves its own; otherwise blocks are transposed and a request covers 32 neighbouring columns of
// a row.  rmax: the lane's row's maximum (ALIGNED) so far.
template <bool ALIGNED>
__device__ __forceinline__ void gated_block32(const GatedParams& p, int row0, int col0, int rows,
                                              int cols, float* g, float* u, bool v8, int lane,
                                              float& rmax) {
  const bool maxima = p.out.row_amax != nullptr || p.out.col_amax != nullptr;
  auto finish = [&] {  // g = act(g) u
    apply_act<32>(p.epi.act, g);
#pragma unroll
    for (int j = 0; j < 32; ++j) g[j] = __fmul_rn(g[j], u[j]);
  };
  auto stored = [&](float v) {  // as D holds it, NaN skipped
    return fmaxf(fabsf(p.d_bf16 ? __bfloat162float(__float2bfloat16_rn(v)) : v), 0.0f);
  };
  if constexpr (ALIGNED) {
    const bool live = lane < rows;
    const int64_t off = (int64_t)(row0 + lane) * p.n + col0;
    if (p.out.gu != nullptr && live) {
      const int64_t at = (int64_t)(row0 + lane) * 2 * p.n + col0;
      store_cols32(p.out.gu, p.d_bf16, at, g, cols, v8);
      store_cols32(p.out.gu, p.d_bf16, at + p.n, u, cols, v8);
    }
    finish();
    if (live) store_cols32(p.d, p.d_bf16, off, g, cols, v8);
    if (!maxima) return;
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      g[j] = live && j < cols ? stored(g[j]) : 0.0f;
      rmax = fmaxf(rmax, g[j]);
    }
    if (p.out.col_amax != nullptr) {
      const float m = lanes_max32(g, lane);
      if (lane < cols) raise(p.out.col_amax + col0 + lane, m);
    }
  } else {
    transpose32(g, lane);  // g[i]: row row0 + i, column col0 + lane
    transpose32(u, lane);
    const bool live = lane < cols;
    auto store = [&](void* base, int64_t at, int64_t pitch, const float* v) {
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        if (!live || i >= rows) continue;
        if (p.d_bf16) static_cast<__nv_bfloat16*>(base)[at + i * pitch] = __float2bfloat16_rn(v[i]);
        else static_cast<float*>(base)[at + i * pitch] = v[i];
      }
    };
    if (p.out.gu != nullptr) {
      const int64_t at = (int64_t)row0 * 2 * p.n + col0 + lane;
      store(p.out.gu, at, 2 * (int64_t)p.n, g);
      store(p.out.gu, at + p.n, 2 * (int64_t)p.n, u);
    }
    finish();
    store(p.d, (int64_t)row0 * p.n + col0 + lane, p.n, g);
    if (!maxima) return;
    float cmax = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      g[i] = live && i < rows ? stored(g[i]) : 0.0f;
      cmax = fmaxf(cmax, g[i]);
    }
    if (p.out.col_amax != nullptr && live) raise(p.out.col_amax + col0 + lane, cmax);
    if (p.out.row_amax != nullptr) {
      const float m = lanes_max32(g, lane);
      if (lane < rows) raise(p.out.row_amax + row0 + lane, m);
    }
  }
}

// ---------------------------------------------------------------- the product

template <bool ALIGNED>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    k_gemm_gated(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                 const GatedParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* factors = reinterpret_cast<float*>(smem + kStages * kStageBytes_);
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(factors) + kFactorBytes);
  uint64_t* empty = full + kStages;
  uint64_t* sf_full = empty + kStages;    // the CTA's scales are in shared memory
  uint64_t* sf_ready = sf_full + kStages;  // the pair's are in tensor memory (the leader's count)
  uint64_t* acc_full = sf_ready + kStages;
  uint64_t* acc_empty = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 1);
  int* err = reinterpret_cast<int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_rank();
  const int pair = blockIdx.x / 2, pairs = gridDim.x / 2;
  const int num_tiles = p.tiles_m * p.tiles_n;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&sf_full[s], 1);
      mbar_init(&sf_ready[s], 2 * kScaleWarps);
    }
    mbar_init(acc_full, 1);
    mbar_init(acc_empty, 2 * kEpilogueWarps);
    *err = 0;
    fence_mbar_init();
    prefetch_tmap(&map_a);
    prefetch_tmap(&map_b);
  }
  if (warp == 1) {
    pair_tmem_alloc(tmem_slot, kTmemCols);
    pair_tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers and tensor memory are there
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp < kScaleWarp0) {
    setmaxnreg_dec<kRegsIssue>();
    if (warp == 0 && lane == 0) {
      // ---------------- producer
      pdl_wait();  // the scales are rewritten
      const uint64_t pol_a = policy_evict_last(), pol_b = policy_evict_normal();
      uint32_t it = 0;  // K tiles issued, over all tiles of this pair
      bool ok = true;
      for (int tile = pair; ok && tile < num_tiles; tile += pairs) {
        int tm, tn;
        tile_at(p, tile, tm, tn);
        const int row = (2 * tm + rank) * kRows, line = rank * p.n + tn * kCols;
        for (int kt = 0; kt < p.k_tiles; ++kt, ++it) {
          const uint32_t s = it % kStages;
          if (it >= (uint32_t)kStages && !mbar_wait_bounded(&empty[s], ((it / kStages) - 1) & 1))
            *err = 1;
          if (*(volatile int*)err) {
            ok = false;
            break;
          }
          uint8_t* st = smem + s * kStageBytes_;
          uint8_t* sf = st + kABytes + kBBytes;
          const uint32_t bar = cluster_addr(&full[s], 0);
          mbar_expect_tx(&sf_full[s], kSfaBytes + kSfbBytes);
          bulk_load(sf, p.sfa + ((int64_t)(2 * tm + rank) * p.k_tiles + kt) * kSfaBytes, kSfaBytes,
                    &sf_full[s], pol_a);
          bulk_load(sf + kSfaBytes, p.sfb + ((int64_t)tn * p.k_tiles + kt) * kSfbBytes, kSfbBytes,
                    &sf_full[s], pol_b);
          if (rank == 0) mbar_expect_tx(&full[s], 2 * (kABytes + kBBytes));
          pair_tma_load_2d(st, &map_a, bar, kt * kKBytes, row, pol_a);
          pair_tma_load_2d(st + kABytes, &map_b, bar, kt * kKBytes, line, pol_b);
        }
      }
      // drain: every copy issued must have landed before the CTAs may exit
      for (uint32_t j = it > (uint32_t)kStages ? it - kStages : 0; j < it; ++j) {
        const uint32_t s = j % kStages, ph = (j / kStages) & 1;
        if (!mbar_wait_bounded(&sf_full[s], ph) || (rank == 0 && !mbar_wait_bounded(&full[s], ph)))
          *err = 1;
      }
    } else if (warp == 1 && lane == 0 && rank == 0) {
      // ---------------- MMA issuer
      uint32_t it = 0, t = 0;
      bool ok = true;
      for (int tile = pair; ok && tile < num_tiles; tile += pairs, ++t) {
        // both CTAs' epilogues of the previous tile have copied the accumulators out
        if (t > 0 && !mbar_wait_bounded(acc_empty, (t - 1) & 1)) {
          *err = 1;
          break;
        }
        tc_fence_after();
        for (int kt = 0; kt < p.k_tiles; ++kt, ++it) {
          const uint32_t s = it % kStages;
          const uint32_t ph = (it / kStages) & 1;
          if (!mbar_wait_bounded(&sf_ready[s], ph) || !mbar_wait_bounded(&full[s], ph)) *err = 1;
          if (*(volatile int*)err) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t st = smem_addr(smem + s * kStageBytes_);
          const uint32_t sfa = tmem + kSfCol0 + s * kSfCols, sfb = sfa + 4 * kKSteps;
#pragma unroll
          for (int ks = 0; ks < kKSteps; ++ks)
            pair_mma_nvf4(tmem, desc_swz128(st + ks * 32), desc_swz128(st + kABytes + ks * 32), p.idesc,
                          sfa + 4 * ks, sfb + 8 * ks, kt != 0 || ks != 0);
          pair_commit(&empty[s]);
        }
        // the accumulators of this tile are complete (or abandoned) once all issued MMAs are
        pair_commit(acc_full);
      }
      // everything issued must be done before TMEM is freed
      if (t > 0 && !mbar_wait_bounded(acc_full, (t - 1) & 1)) *err = 1;
    }
  } else if (warp < kEpilogueWarp0) {
    setmaxnreg_dec<kRegsScales>();
    // ---------------- scales: lane l of a quarter holds the words of lines l, l + 32, ... of a
    // piece, the same in every quarter
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const int tiles = (num_tiles - pair + pairs - 1) / pairs;
    const uint32_t all = (uint32_t)tiles * p.k_tiles;
    for (uint32_t it = 0; it < all; ++it) {
      const uint32_t s = it % kStages, ph = (it / kStages) & 1;
      // (the producer refills the stage only when the MMAs that read the slot are done)
      bool ok = mbar_wait_bounded(&sf_full[s], ph);
      if (!ok) *err = 1;
      if (__any_sync(0xffffffffu, !ok || *(volatile int*)err)) break;
      tc_fence_after();
      const uint4* from = reinterpret_cast<const uint4*>(smem + s * kStageBytes_ + kABytes + kBBytes) + lane;
      const uint32_t sf = tmem + lanes + kSfCol0 + s * kSfCols;
      uint32_t w[3][16];
#pragma unroll
      for (int c = 0; c < 3; ++c)
#pragma unroll
        for (int ks = 0; ks < kKSteps; ++ks) {
          // columns: A's K steps; B's by K step, the gate's lines and then up's
          const int piece = c == 0 ? ks : kKSteps * (1 + (ks & 1)) + 2 * (c - 1) + (ks >> 1);
          const uint4 v = from[piece * (kPiece / 16)];
          w[c][4 * ks] = v.x, w[c][4 * ks + 1] = v.y, w[c][4 * ks + 2] = v.z, w[c][4 * ks + 3] = v.w;
        }
#pragma unroll
      for (int c = 0; c < 3; ++c) tmem_st16(sf + 16 * c, w[c]);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) cluster_arrive(cluster_addr(&sf_ready[s], 0));
    }
  } else {
    setmaxnreg_inc<kRegsEpilogue>();
    // ---------------- epilogue: lane quarter q (rows 32q ..), column half `half`
    const int q = warp & 3, half = (warp - kEpilogueWarp0) >> 2;
    float* beta = factors + (warp - kEpilogueWarp0) * 4 * kWarpCols;  // [gate, up][64], then their bias
    float* bias = beta + 2 * kWarpCols;
    const uint32_t hand_back = cluster_addr(acc_empty, 0);
    const bool v8 = (alignment(p) & 31) == 0;
    bool cleared = false;
    uint32_t t = 0;
    for (int tile = pair; tile < num_tiles; tile += pairs, ++t) {
      int tm, tn;
      tile_at(p, tile, tm, tn);
      const int row0 = (2 * tm + rank) * kRows + q * 32;
      const int col0 = tn * kCols + half * kWarpCols;
      const int rows = min(32, p.m - row0), cols = min(kWarpCols, p.n - col0);
      // before the accumulators are ready: the row factor alpha = fl(amax_a[row] fl(1/F_a)),
      // the column factors beta and the bias, lane l those of columns 2l, 2l + 1 of each half
      const float alpha =
          lane < rows ? __fmul_rn(__ldg(p.a_amax + (int64_t)(row0 + lane) * p.a_amax_stride), p.a_finv)
                      : 0.0f;
      __syncwarp();  // every lane has read the previous tile's factors
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int c = 2 * lane + j, line = h * p.n + col0 + c;
          const bool in = c < cols;
          beta[h * kWarpCols + c] =
              in ? __fmul_rn(__ldg(p.b_amax + (int64_t)line * p.b_amax_stride), p.b_finv) : 0.0f;
          bias[h * kWarpCols + c] = p.epi.bias_at(in ? line : -1);
        }
      __syncwarp();
      const bool ready = mbar_wait_bounded(acc_full, t & 1);
      if (!ready) *err = 1;
      tc_fence_after();
      // All accumulators at once, so that TMEM may take the next tile's MMAs during the rest; rows
      // that are not aligned have no registers for that beside their transpositions (4 bytes of
      // spills a value, measured twice as slow; 28 bytes in all are left), and hand TMEM back after their
      // last block.
      constexpr int kHeld = ALIGNED ? kWarpCols : 32;
      uint32_t v[2][kHeld];
      auto load = [&](int from) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int c = 0; c < kHeld; c += 32)
            tmem_ld32(tmem + ((uint32_t)(q * 32) << 16) + h * kCols + half * kWarpCols + from + c,
                      v[h] + c);
        tmem_ld_wait();
        if (from + kHeld < kWarpCols) return;
        tc_fence_before();
        __syncwarp();
        if (lane == 0) cluster_arrive(hand_back);
      };
      load(0);
      // the warp leaves together: what follows (shuffles, the next tile's TMEM loads) takes
      // every lane, and each lane's wait gives up by its own clock
      if (__any_sync(0xffffffffu, !ready || *(volatile int*)err)) break;
      if (!cleared && (p.out.row_amax != nullptr || p.out.col_amax != nullptr)) pdl_wait();
      cleared = true;
      float rmax = 0.0f;
#pragma unroll
      for (int c = 0; c < kWarpCols; c += 32) {
        if (c > 0 && !ALIGNED) load(c);
        if (rows <= 0 || c >= cols) continue;
        float z[2][32];
        // fl(fl(acc * alpha) * beta) + bias
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j4 = 0; j4 < 32; j4 += 4) {
            const float4 b4 = *reinterpret_cast<const float4*>(beta + h * kWarpCols + c + j4);
            const float4 a4 = *reinterpret_cast<const float4*>(bias + h * kWarpCols + c + j4);
            const float bj[4] = {b4.x, b4.y, b4.z, b4.w}, aj[4] = {a4.x, a4.y, a4.z, a4.w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              z[h][j4 + j] = __fadd_rn(
                  __fmul_rn(__fmul_rn(__uint_as_float(v[h][c % kHeld + j4 + j]), alpha), bj[j]),
                  aj[j]);
          }
        gated_block32<ALIGNED>(p, row0, col0 + c, rows, min(32, cols - c), z[0], z[1], v8, lane, rmax);
      }
      if (ALIGNED && p.out.row_amax != nullptr && lane < rows) raise(p.out.row_amax + row0 + lane, rmax);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (threadIdx.x == 0 && *(volatile int*)err) raise_status(p.status, kStatusTimeout);
  __syncwarp();
  cluster_sync();  // nothing of either CTA is used by the other any more
  if (warp == 1) {
    tc_fence_after();
    pair_tmem_dealloc(tmem, kTmemCols);
  }
}

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Layout {
  int64_t k_tiles, tiles_m, tiles_n, a_bytes, bytes;
  Layout(int64_t m, int64_t n, int64_t k)
      : k_tiles(ceil_div(k, 2 * kKBytes)), tiles_m(ceil_div(m, 2 * kRows)),
        tiles_n(ceil_div(n, kCols)), a_bytes(2 * tiles_m * k_tiles * kSfaBytes),
        bytes(a_bytes + 2 * tiles_n * k_tiles * kSfaBytes) {}
};

template <bool ALIGNED>
cudaError_t run(const CUtensorMap& map_a, const CUtensorMap& map_b, const GatedParams& p,
                int64_t tiles, const DeviceInfo& dev, cudaStream_t stream) {
  const auto kernel = k_gemm_gated<ALIGNED>;
  // clusters that are resident at once, by device (0: not asked yet).  Threads that make their first calls
  // at once all ask; who reads a count also has the attribute that was set before it
  static std::atomic<int> pairs_of[64];
  int pairs = dev.device < 64 ? pairs_of[dev.device].load(std::memory_order_acquire) : 0;
  if (pairs == 0) {
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         kSmemBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2 * (dev.num_sms / 2));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cudaLaunchAttribute at{};
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = 2;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&pairs, kernel, &cfg);
    if (e != cudaSuccess) return e;
    if (pairs < 1) return cudaErrorInvalidConfiguration;
    if (dev.device < 64) pairs_of[dev.device].store(pairs, std::memory_order_release);
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(2 * std::min<int64_t>(tiles, pairs)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmemBytes;
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, map_a, map_b, p);
}

}  // namespace

int64_t gemm_gated_workspace(int64_t m, int64_t n, int64_t k) { return Layout(m, n, k).bytes; }

cudaError_t launch_gemm_gated(const GemmArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  const Layout L(a.M, a.N, a.K);
  uint8_t* sf = a.workspace;
  CUtensorMap map_a, map_b;
  if (!make_operand_map(&map_a, a.a_codes, a.M, a.K / 2, kKBytes, kRows) ||
      !make_operand_map(&map_b, a.b_codes, 2 * a.N, a.K / 2, kKBytes, kCols))
    return cudaErrorInvalidValue;
  ScaleArgs s{a.a_scales, a.b_scales, a.M, a.N, a.K / 16, (int)L.k_tiles, (int)(2 * L.tiles_m),
              (int)(2 * L.tiles_n), sf, a.gated->row_amax, a.gated->col_amax};
  const int64_t ctas =
      (int64_t)(s.a_blocks + s.b_blocks) * ceil_div(L.k_tiles, kScaleTiles);
  k_gated_scales<<<(unsigned)ctas, 256, 0, stream>>>(s);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  GatedParams p{};
  p.sfa = sf;
  p.sfb = sf + L.a_bytes;
  p.a_amax = a.a_amax;
  p.b_amax = a.b_amax;
  p.a_amax_stride = a.a_row_scaled ? 1 : 0;
  p.b_amax_stride = a.b_row_scaled ? 1 : 0;
  p.a_finv = 1.0f / (a.a_bound * 6.0f);
  p.b_finv = 1.0f / (a.b_bound * 6.0f);
  p.m = (int)a.M;
  p.n = (int)a.N;
  p.k_tiles = (int)L.k_tiles;
  p.tiles_m = (int)L.tiles_m;
  p.tiles_n = (int)L.tiles_n;
  p.d = a.d;
  p.d_bf16 = a.d_bf16;
  p.epi = *a.epilogue;
  p.out = *a.gated;
  p.idesc = make_idesc_nvf4(2 * kRows, 2 * kCols);
  p.status = dev.status;
  const int64_t tiles = L.tiles_m * L.tiles_n;
  return alignment(p) % 16 == 0 ? run<true>(map_a, map_b, p, tiles, dev, stream)
                                : run<false>(map_a, map_b, p, tiles, dev, stream);
}

}  // namespace nvfp4
