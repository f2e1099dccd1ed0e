// kernels_gemm_few.cu -- the NVFP4 product with its epilogue for few rows of A (decoded
// tokens): D [m][n] = act(A B^T + bias) + residual, m <= 128.
//
// With few rows the product reads B (the weights) once and is bound by that: 0.5625 bytes
// per weight.  So the roles are exchanged: 128 lines of B are the MMA's M, the m rows of
// A (padded to 16, 32, 64 or 128) its N, and what has to be right is the stream of B:
//   * the work is cut into units of 128 lines x 256 values, numbered along K first, and
//     every SM's CTA takes an equal run of them, so all SMs stream to the end whatever n
//     and k are; a tile of 128 lines that two or more CTAs share is joined by the CTA
//     that finishes it last, from partial sums in the workspace, added in the CTAs' order
//     (the result does not depend on which one that is);
//   * the compact scales are read as they lie (no pass over them beforehand): a line's 16
//     scale bytes of a unit are one load of one thread, kPrefetch units ahead, and go
//     from registers straight into tensor memory.
// Warps: 0 loads codes (TMA, a ring of S stages), 1 issues the MMAs, 2-5 write scales to
// TMEM (one per lane quarter), 6-9 are the epilogue (two accumulators, so the next tile's
// MMAs run meanwhile).  Lane l of the accumulator is line l of B, so a warp writes 32
// neighbouring columns of D for each row.
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
constexpr int kUnitBytes = 128; // code bytes of a line per unit: 256 values
constexpr int kUnitScales = 16;
constexpr int kPrefetch = 4;    // units whose scales are in registers ahead
constexpr int kFewThreads = 320;
constexpr int kMaxCtas = 256;   // bound of the grid, for the workspace

struct FewParams {
  const uint8_t* x_scales;
  const uint8_t* w_scales;
  int x_grain, w_grain;  // widest access of the scale rows: 16, 4, 2 or 1 bytes
  const float* x_amax;
  const float* w_amax;
  int x_amax_stride, w_amax_stride;
  float x_finv, w_finv;
  int m, n;
  int64_t k16;      // scales per line
  int k_tiles;      // units per tile
  int64_t units;    // all units
  void* d;
  bool d_bf16;
  Epilogue epi;
  uint32_t* arrivals;  // [tiles], zero before the kernel's first arrival
  float* part;         // [gridDim.x][2][NT][128] partial sums
  uint32_t idesc;
  int* status;
};

// Up to 16 scale bytes at p as four words, zero from n on.
__device__ __forceinline__ void load_scales(const uint8_t* p, int n, int grain, uint32_t* w) {
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = 0;
  if (n <= 0) return;
  if (grain == 16) {  // n is 16
    const uint4 v = __ldg(reinterpret_cast<const uint4*>(p));
    w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
  } else if (grain == 4) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (4 * j < n) w[j] = __ldg(reinterpret_cast<const uint32_t*>(p) + j);
  } else if (grain == 2) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (2 * j < n)
        w[j >> 1] |= (uint32_t)__ldg(reinterpret_cast<const uint16_t*>(p) + j) << (16 * (j & 1));
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j)
      if (j < n) w[j >> 2] |= (uint32_t)__ldg(p + j) << (8 * (j & 3));
  }
}

// Named barrier 1 over the four epilogue warps, with the OR of a flag.
__device__ __forceinline__ bool epilogue_barrier_or(bool flag) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 128, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"((uint32_t)flag)
      : "memory");
  return any != 0;
}

__device__ __forceinline__ int64_t first_unit(int64_t units, int ctas, int cta) {
  return units * cta / ctas;
}
__device__ __forceinline__ int cta_of_unit(int64_t units, int ctas, int64_t u) {
  return (int)(((u + 1) * ctas - 1) / units);
}

// One element: the scaled sum (as in kernels_gemm.cu), the epilogue, the store.
__device__ __forceinline__ void few_store(const FewParams& p, int row, int col, float acc,
                                          float beta, float bias) {
  const float alpha = __fmul_rn(__ldg(p.x_amax + (int64_t)row * p.x_amax_stride), p.x_finv);
  float v = __fadd_rn(__fmul_rn(__fmul_rn(acc, alpha), beta), bias);
  const int64_t at = (int64_t)row * p.n + col;
  if (p.epi.z != nullptr) {
    if (p.d_bf16) static_cast<__nv_bfloat16*>(p.epi.z)[at] = __float2bfloat16_rn(v);
    else static_cast<float*>(p.epi.z)[at] = v;
  }
  if (p.epi.act == kActRelu) v = act_value<kActRelu>(v);
  else if (p.epi.act == kActGelu) v = act_value<kActGelu>(v);
  else if (p.epi.act == kActSilu) v = act_value<kActSilu>(v);
  if (p.epi.residual != nullptr)
    v = __fadd_rn(v, p.d_bf16
                         ? __bfloat162float(static_cast<const __nv_bfloat16*>(p.epi.residual)[at])
                         : static_cast<const float*>(p.epi.residual)[at]);
  if (p.d_bf16) static_cast<__nv_bfloat16*>(p.d)[at] = __float2bfloat16_rn(v);
  else static_cast<float*>(p.d)[at] = v;
}

// NT: rows of A per MMA (its N); S: stages of the code ring and of the TMEM scale slots.
template <int NT, int S>
struct FewGeom {
  static constexpr int kABytes = kLines * kUnitBytes;
  static constexpr int kStageBytes = kABytes + NT * kUnitBytes;
  static constexpr int kSmemBytes = S * kStageBytes + 1024 /* alignment */ + 512 /* barriers */;
  static constexpr int kSfCol0 = 2 * NT;  // two accumulators, then 32 columns per slot
  static constexpr int kTmemCols = 512;
  static_assert(kSfCol0 + 32 * S <= kTmemCols, "TMEM columns");
  static_assert(kStageBytes % 1024 == 0, "128B swizzle");
  static_assert(kSmemBytes <= 232448, "shared memory");
};

template <int NT, int S>
__global__ void __launch_bounds__(kFewThreads, 1)
    k_gemm_few(const __grid_constant__ CUtensorMap map_w, const __grid_constant__ CUtensorMap map_x,
               const FewParams p) {
  using G = FewGeom<NT, S>;
  constexpr int kXGroups = (NT + 31) / 32;  // 32-row groups of A: TMEM columns of its scales
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + S * G::kStageBytes);
  uint64_t* empty = full + S;
  uint64_t* sf_full = empty + S;
  uint64_t* acc_full = sf_full + S;
  uint64_t* acc_empty = acc_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(acc_empty + 2);
  int* err = reinterpret_cast<int*>(tmem_slot + 1);
  int* last_flag = err + 1;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t u0 = first_unit(p.units, gridDim.x, blockIdx.x);
  const int64_t u1 = first_unit(p.units, gridDim.x, blockIdx.x + 1);

  if (threadIdx.x == 0) {
    for (int s = 0; s < S; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&sf_full[s], 4);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 4);
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
    int tile = (int)(u0 / p.k_tiles), kt = (int)(u0 % p.k_tiles);
    for (int64_t u = u0; u < u1; ++u, ++it) {
      const uint32_t s = it % S;
      if (it >= (uint32_t)S && !mbar_wait_bounded(&empty[s], ((it / S) - 1) & 1)) {
        *err = 1;
        break;
      }
      if (*(volatile int*)err) break;
      uint8_t* st = smem + s * G::kStageBytes;
      mbar_expect_tx(&full[s], G::kStageBytes);
      tma_load_2d(st, &map_w, &full[s], kt * kUnitBytes, tile * kLines, pol_w);
      tma_load_2d(st + G::kABytes, &map_x, &full[s], kt * kUnitBytes, 0, pol_x);
      if (++kt == p.k_tiles) {
        kt = 0;
        ++tile;
      }
    }
    // every copy issued must have landed before the CTA may exit
    for (uint32_t j = it > (uint32_t)S ? it - S : 0; j < it; ++j)
      if (!mbar_wait_bounded(&full[j % S], (j / S) & 1)) *err = 1;
  } else if (warp == 1 && lane == 0) {
    // ---------------- MMAs: four per unit, one accumulator per tile of the run
    uint32_t it = 0, seg = 0;
    bool ok = true;
    for (int64_t u = u0; ok && u < u1; ++seg) {
      const int64_t end = min(u1, (u / p.k_tiles + 1) * p.k_tiles);
      const uint32_t b = seg & 1;
      if (seg >= 2 && !mbar_wait_bounded(&acc_empty[b], ((seg >> 1) - 1) & 1)) {
        *err = 1;
        break;
      }
      tc_fence_after();
      for (bool first = true; u < end; ++u, ++it, first = false) {
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
        const uint32_t sf = tmem + G::kSfCol0 + 32 * s;
#pragma unroll
        for (int ks = 0; ks < 4; ++ks)
          tc_mma_nvf4(tmem + b * NT, desc_swz128(st + 32 * ks),
                      desc_swz128(st + G::kABytes + 32 * ks), p.idesc, sf + 4 * ks,
                      sf + 16 + 4 * ks, !first || ks != 0);
        tc_commit(&empty[s]);
      }
      tc_commit(&acc_full[b]);
    }
    // everything issued must be done before TMEM is freed
    for (uint32_t j = seg > 2 ? seg - 2 : 0; j < seg; ++j)
      if (!mbar_wait_bounded(&acc_full[j & 1], (j >> 1) & 1)) *err = 1;
  } else if (warp >= 2 && warp < 6) {
    // ---------------- scales: lane quarter q holds the B lines 32q + lane, and a copy of
    // the scales of all rows of A
    const int q = warp & 3;
    uint32_t wa[kPrefetch][4], wb[kPrefetch][kXGroups][4];
    int tile = (int)(u0 / p.k_tiles), kt = (int)(u0 % p.k_tiles);  // of the next load
    const int64_t count = u1 - u0;
    auto fetch = [&](int slot) {
      const int64_t s0 = (int64_t)kt * kUnitScales;
      const int n = (int)min((int64_t)kUnitScales, p.k16 - s0);
      const int line = tile * kLines + 32 * q + lane;
      load_scales(p.w_scales + line * p.k16 + s0, line < p.n ? n : 0, p.w_grain, wa[slot]);
#pragma unroll
      for (int c = 0; c < kXGroups; ++c) {
        const int row = 32 * c + lane;
        load_scales(p.x_scales + row * p.k16 + s0, row < p.m ? n : 0, p.x_grain, wb[slot][c]);
      }
      if (++kt == p.k_tiles) {
        kt = 0;
        ++tile;
      }
    };
#pragma unroll
    for (int j = 0; j < kPrefetch; ++j)
      if (j < count) fetch(j);
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    bool ok = true;
    for (int64_t base = 0; ok && base < count; base += kPrefetch) {
#pragma unroll
      for (int j = 0; j < kPrefetch; ++j) {
        const int64_t i = base + j;
        if (!ok || i >= count) break;
        const uint32_t it = (uint32_t)i, s = it % S;
        if (it >= (uint32_t)S) ok = mbar_wait_bounded(&empty[s], ((it / S) - 1) & 1);
        ok = __all_sync(0xffffffffu, ok && !*(volatile int*)err);
        if (!ok) {
          *err = 1;
          break;
        }
        tc_fence_after();
        const uint32_t sf = tmem + lanes + G::kSfCol0 + 32 * s;
        uint32_t r[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) r[e] = wa[j][e >> 2];  // read at column q of each four
        tmem_st16(sf, r);
#pragma unroll
        for (int e = 0; e < 16; ++e)
          r[e] = (e & 3) < kXGroups ? wb[j][(e & 3) < kXGroups ? (e & 3) : 0][e >> 2] : 0u;
        tmem_st16(sf + 16, r);
        if (i + kPrefetch < count) fetch(j);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sf_full[s]);
      }
    }
  } else if (warp >= 6) {
    // ---------------- epilogue
    const int q = warp & 3, l = 32 * q + lane;
    const uint32_t lanes = (uint32_t)(q * 32) << 16;
    uint32_t seg = 0;
    for (int64_t u = u0; u < u1; ++seg) {
      const int tile = (int)(u / p.k_tiles);
      const int64_t t0 = (int64_t)tile * p.k_tiles, t1 = t0 + p.k_tiles;
      const int64_t end = min(u1, t1);
      const bool whole = u == t0 && end == t1;
      u = end;
      const uint32_t b = seg & 1;
      const int col = tile * kLines + l;
      const bool live = col < p.n;
      float beta = 0.0f, bias = 0.0f;
      if (live) {
        beta = __fmul_rn(__ldg(p.w_amax + (int64_t)col * p.w_amax_stride), p.w_finv);
        bias = p.epi.bias_at(col);
      }
      const bool ready = mbar_wait_bounded(&acc_full[b], (seg >> 1) & 1);
      if (!ready) *err = 1;
      if (epilogue_barrier_or(!ready || *(volatile int*)err)) break;
      tc_fence_after();
      // this CTA's partial sums of the tile: slot 0 for its first tile, 1 for its last
      float* part = p.part + ((int64_t)blockIdx.x * 2 + (seg == 0 ? 0 : 1)) * NT * kLines + l;
#pragma unroll 1
      for (int c = 0; c < NT; c += 16) {
        if (c >= p.m) break;
        uint32_t v[16];
        tmem_ld16(tmem + lanes + b * NT + c, v);
        tmem_ld_wait();
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          if (c + j >= p.m) break;
          if (!whole) __stcg(part + (c + j) * kLines, __uint_as_float(v[j]));
          else if (live) few_store(p, c + j, col, __uint_as_float(v[j]), beta, bias);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&acc_empty[b]);
      if (whole) continue;
      // the tile's last CTA adds all partial sums, in the CTAs' order
      __threadfence();
      epilogue_barrier_or(false);
      const int c0 = cta_of_unit(p.units, gridDim.x, t0);
      const int c1 = cta_of_unit(p.units, gridDim.x, t1 - 1);
      if (warp == 6 && lane == 0) {
        pdl_wait();  // the arrival counts are zero
        *last_flag = atomicAdd(p.arrivals + tile, 1u) == (uint32_t)(c1 - c0);
        __threadfence();
      }
      epilogue_barrier_or(false);
      const bool last = *(volatile int*)last_flag != 0;
      epilogue_barrier_or(false);  // read before it is written again
      if (!last || !live) continue;
      for (int j = 0; j < p.m; ++j) {
        float sum = 0.0f;
        for (int c = c0; c <= c1; ++c) {
          const int slot = first_unit(p.units, gridDim.x, c) >= t0 ? 0 : 1;
          const float* from = p.part + (((int64_t)c * 2 + slot) * NT + j) * kLines + l;
          sum = c == c0 ? __ldcg(from) : __fadd_rn(sum, __ldcg(from));
        }
        few_store(p, j, col, sum, beta, bias);
      }
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

// Clears the arrival counts.  The product starts while this runs (it needs the counts only
// at its first shared tile).
__global__ void k_clear_arrivals(uint32_t* p, int n) {
  pdl_launch_dependents();
  for (int i = threadIdx.x; i < n; i += blockDim.x) p[i] = 0;
}

int scale_grain(const uint8_t* p, int64_t k16) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p) | (uintptr_t)k16;
  return a % 16 == 0 ? 16 : (a % 4 == 0 ? 4 : (a % 2 == 0 ? 2 : 1));
}

int rows_of_mma(int64_t m) { return m <= 16 ? 16 : (m <= 32 ? 32 : (m <= 64 ? 64 : 128)); }
int64_t tiles_of(int64_t n) { return (n + kLines - 1) / kLines; }
int64_t round256(int64_t v) { return (v + 255) / 256 * 256; }

template <int NT, int S>
cudaError_t run_few(const GemmArgs& a, FewParams& p, const CUtensorMap& map_w,
                    const CUtensorMap& map_x, int grid, bool shared_tiles, int tiles,
                    cudaStream_t stream) {
  using G = FewGeom<NT, S>;
  auto kernel = k_gemm_few<NT, S>;
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
  if (shared_tiles) {
    k_clear_arrivals<<<1, 256, 0, stream>>>(p.arrivals, tiles);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, kernel, map_w, map_x, p);
}

}  // namespace

bool gemm_few_rows(int64_t m) { return m <= kGemmFewRows; }

int64_t gemm_few_workspace(int64_t m, int64_t n) {
  return round256(4 * tiles_of(n)) + (int64_t)kMaxCtas * 2 * rows_of_mma(m) * kLines * 4;
}

cudaError_t launch_gemm_few(const GemmArgs& a, const DeviceInfo& dev, cudaStream_t stream) {
  const int nt = rows_of_mma(a.M);
  CUtensorMap map_w, map_x;
  if (!make_operand_map(&map_w, a.b_codes, a.N, a.K / 2, kUnitBytes, kLines) ||
      !make_operand_map(&map_x, a.a_codes, a.M, a.K / 2, kUnitBytes, nt))
    return cudaErrorInvalidValue;
  const int tiles = (int)tiles_of(a.N);
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
  p.k_tiles = (int)((a.K + 2 * kUnitBytes - 1) / (2 * kUnitBytes));
  p.units = (int64_t)tiles * p.k_tiles;
  p.d = a.d;
  p.d_bf16 = a.d_bf16;
  p.epi = *a.epilogue;
  p.arrivals = reinterpret_cast<uint32_t*>(a.workspace);
  p.part = reinterpret_cast<float*>(a.workspace + round256(4 * (int64_t)tiles));
  p.status = dev.status;
  // at least four units a CTA: below that the joining costs more than the CTA adds
  const int most = std::min(dev.num_sms, kMaxCtas);
  const int grid = (int)std::max<int64_t>(1, std::min<int64_t>(most, (p.units + 3) / 4));
  const bool shared_tiles = p.units % grid != 0 || (p.units / grid) % p.k_tiles != 0;
  switch (nt) {
    case 16: return run_few<16, 11>(a, p, map_w, map_x, grid, shared_tiles, tiles, stream);
    case 32: return run_few<32, 10>(a, p, map_w, map_x, grid, shared_tiles, tiles, stream);
    case 64: return run_few<64, 8>(a, p, map_w, map_x, grid, shared_tiles, tiles, stream);
    default: return run_few<128, 6>(a, p, map_w, map_x, grid, shared_tiles, tiles, stream);
  }
}

}  // namespace nvfp4
