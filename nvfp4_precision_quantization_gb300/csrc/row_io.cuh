// row_io.cuh -- 16 consecutive row elements per thread: loads and stores shared by the
// layer operators' kernels (BF16 or FP32 rows, widened to FP32).
//
// A row may start at any element.  `grain` is the widest access that every row of the tensor
// allows, the same for the whole tensor, so the choice is one uniform branch.  32- and
// 16-byte accesses are made by each lane on its own chunk (a row's last chunk, cut by its
// end, element by element).  Narrower ones would make every request of a warp touch 32
// sectors, so there the warp moves its 32 chunks together: neighbouring lanes access
// neighbouring units of 8, 4, 2 or 1 bytes, and 1 KB of shared memory per warp turns that
// into whole chunks per lane and back (5001 columns instead of 5000 measured 7 times slower
// without it).
#pragma once

#include <cuda_bf16.h>

#include "device_common.cuh"

namespace nvfp4 {

constexpr int kChunk = 16;  // elements per thread and access group

// Launch a kernel whose set-up may overlap the end of the one before it in the stream; it
// begins with pdl_wait().
template <typename... P>
inline cudaError_t launch_after(void (*kernel)(P...), unsigned grid, unsigned threads,
                                cudaStream_t stream, const P&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cudaLaunchAttribute at{};
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// The grain of rows of `bytes` bytes at p: 32, 16, 8, 4, 2 or 1.
inline int row_grain(const void* p, int64_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p) | (uintptr_t)bytes;
  int g = 32;
  while (a % g != 0) g /= 2;
  return g;
}

constexpr int kStageBytes = 1024;  // of shared memory per warp

// Staged accesses of a warp: W words per lane (at most 8), lanes PITCH bytes apart from lane
// 0's first byte, of which the first `bytes` bytes of the whole run exist.  Unit i of the
// warp's 32 W / unit is byte i * unit % (4 W) of lane i * unit / (4 W).
template <int W, int PITCH, int UNIT>
struct StagedUnits {
  static constexpr int kPer = 4 * W / UNIT;  // units per lane
  static constexpr int kAll = 31 * PITCH + 4 * W;  // the bytes of a whole run
  static_assert(W <= 8 && 4 * W * 32 <= kStageBytes, "one pass");
  __device__ __forceinline__ static int at(int i, int lane) { return (32 * i + lane) * UNIT; }
  __device__ __forceinline__ static int offset(int i, int lane) {
    if constexpr (PITCH == 4 * W) return at(i, lane);
    // a step of i is 32 units: a whole number of lanes
    static_assert(32 * UNIT % (4 * W) == 0, "units of a step");
    return (lane * UNIT) / (4 * W) * PITCH + (lane * UNIT) % (4 * W) +
           i * (32 * UNIT / (4 * W)) * PITCH;
  }
};
template <int UNIT>
struct UnitType;
template <>
struct UnitType<8> {
  using type = uint2;
};
template <>
struct UnitType<4> {
  using type = uint32_t;
};
template <>
struct UnitType<2> {
  using type = uint16_t;
};
template <>
struct UnitType<1> {
  using type = uint8_t;
};

// A staged load in two steps, so that several can be in flight: the warp's units into
// registers, then through shared memory into each lane's W words.  ELEM: bytes of an element,
// the least unit that there can be.
template <int W, int PITCH, int ELEM>
struct StagedLoad {
  uint32_t v[2 * W];  // units of 2 bytes take a register each, wider ones W words in all

  template <int UNIT, bool WHOLE>
  __device__ __forceinline__ void issue_units(const char* p, int bytes, int lane) {
    using U = StagedUnits<W, PITCH, UNIT>;
    using T = typename UnitType<UNIT>::type;
#pragma unroll
    for (int i = 0; i < U::kPer; ++i) {
      const int off = U::offset(i, lane);
      const T t = WHOLE || off < bytes ? *reinterpret_cast<const T*>(p + off) : T{};
      if constexpr (UNIT == 8) {
        v[2 * i] = t.x;
        v[2 * i + 1] = t.y;
      } else {
        v[i] = t;
      }
    }
  }
  template <int UNIT>
  __device__ __forceinline__ void issue_units(const char* p, int bytes, int lane) {
    if (bytes >= StagedUnits<W, PITCH, UNIT>::kAll) issue_units<UNIT, true>(p, bytes, lane);
    else issue_units<UNIT, false>(p, bytes, lane);
  }
  template <int UNIT>
  __device__ __forceinline__ void settle_units(uint8_t* smem, int lane) const {
    using U = StagedUnits<W, PITCH, UNIT>;
    using T = typename UnitType<UNIT>::type;
#pragma unroll
    for (int i = 0; i < U::kPer; ++i) {
      T* to = reinterpret_cast<T*>(smem + U::at(i, lane));
      if constexpr (UNIT == 8) *to = make_uint2(v[2 * i], v[2 * i + 1]);
      else *to = (T)v[i];
    }
  }
  __device__ __forceinline__ void issue(const char* p, int bytes, int unit, int lane) {
    if (unit == 8) issue_units<8>(p, bytes, lane);
    else if (ELEM == 4 || unit == 4) issue_units<4>(p, bytes, lane);
    else if constexpr (ELEM == 2) issue_units<2>(p, bytes, lane);
  }
  __device__ __forceinline__ void settle(int unit, uint8_t* smem, int lane, uint32_t* w) const {
    if (unit == 8) settle_units<8>(smem, lane);
    else if (ELEM == 4 || unit == 4) settle_units<4>(smem, lane);
    else if constexpr (ELEM == 2) settle_units<2>(smem, lane);
    __syncwarp();
#pragma unroll
    for (int k = 0; k < W; k += 4) {
      const uint4 u = *reinterpret_cast<const uint4*>(smem + 4 * W * lane + 4 * k);
      w[k] = u.x, w[k + 1] = u.y, w[k + 2] = u.z, w[k + 3] = u.w;
    }
    __syncwarp();
  }
};

template <int W, int PITCH, int UNIT, bool WHOLE>
__device__ __forceinline__ void staged_store_units(char* p, int bytes, const uint8_t* smem,
                                                   int lane) {
  using U = StagedUnits<W, PITCH, UNIT>;
  using T = typename UnitType<UNIT>::type;
#pragma unroll
  for (int i = 0; i < U::kPer; ++i) {
    const int off = U::offset(i, lane);
    if (WHOLE || off < bytes)
      *reinterpret_cast<T*>(p + off) = *reinterpret_cast<const T*>(smem + U::at(i, lane));
  }
}
template <int W, int PITCH, int UNIT>
__device__ __forceinline__ void staged_store_units(char* p, int bytes, const uint8_t* smem,
                                                   int lane) {
  if (bytes >= StagedUnits<W, PITCH, UNIT>::kAll)
    staged_store_units<W, PITCH, UNIT, true>(p, bytes, smem, lane);
  else
    staged_store_units<W, PITCH, UNIT, false>(p, bytes, smem, lane);
}
template <int W, int PITCH, int LEAST, int MOST>
__device__ __forceinline__ void staged_store_least(char* p, int bytes, int unit,
                                                   const uint8_t* smem, int lane) {
  if constexpr (MOST > LEAST) {
    if (unit < MOST) {
      staged_store_least<W, PITCH, LEAST, MOST / 2>(p, bytes, unit, smem, lane);
      return;
    }
  }
  staged_store_units<W, PITCH, MOST>(p, bytes, smem, lane);
}
// Words of every lane to memory through shared memory (see StagedUnits), in units of LEAST to
// MOST bytes.
template <int W, int PITCH, int LEAST, int MOST>
__device__ __forceinline__ void staged_store(char* p, int bytes, int unit, uint8_t* smem,
                                             int lane, const uint32_t* w) {
  if constexpr (W % 4 == 0) {
#pragma unroll
    for (int k = 0; k < W; k += 4)
      *reinterpret_cast<uint4*>(smem + 4 * W * lane + 4 * k) =
          make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
  } else {
#pragma unroll
    for (int k = 0; k < W; ++k)
      *reinterpret_cast<uint32_t*>(smem + 4 * W * lane + 4 * k) = w[k];
  }
  __syncwarp();
  staged_store_least<W, PITCH, LEAST, MOST>(p, bytes, unit, smem, lane);
  __syncwarp();
}

// Bytes [at, at + d) of a unit (at a multiple of d; d: 1, 2, 4 or 8) to q + at.
__device__ __forceinline__ void store_piece(char* q, const uint32_t* x, int at, int d) {
  if (d == 8) {
    *reinterpret_cast<uint2*>(q + at) = at & 8 ? make_uint2(x[2], x[3]) : make_uint2(x[0], x[1]);
    return;
  }
  const uint32_t hi = at & 4 ? x[3] : x[2], lo = at & 4 ? x[1] : x[0], w = at & 8 ? hi : lo;
  if (d == 4) *reinterpret_cast<uint32_t*>(q + at) = w;
  else if (d == 2) *reinterpret_cast<uint16_t*>(q + at) = (uint16_t)(w >> (8 * (at & 2)));
  else *reinterpret_cast<uint8_t*>(q + at) = (uint8_t)(w >> (8 * (at & 3)));
}

// 16 one-byte codes of every lane, at most `bytes` bytes in all, to memory from any byte p on
// as aligned 16-byte units: each lane takes the words of the lane before it and shifts its own
// behind them, so that what it holds starts on a unit.  The units that the run begins and ends
// in are stored as pieces of 1 to 8 bytes.  (The staging makes 16 one-byte stores of it: 4000
// x 5001 norm 69 us that way, 58 this way.  For 2- and 4-byte elements, whose staging needs
// half and a quarter of the stores, the shifts cost more than they save: 16384 x 1001 41 us
// staged, 45 shifted.)
__device__ __forceinline__ void shifted_store(char* p, int bytes, int lane, const uint32_t* w) {
  constexpr int W = 4;
  if (bytes <= 0) return;  // the same for the whole warp
  const int b = (int)(reinterpret_cast<uintptr_t>(p) & 15);
  uint32_t z[W + 8];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    z[k] = __shfl_up_sync(0xffffffffu, w[W - 4 + k], 1);
    z[W + 4 + k] = 0;
  }
#pragma unroll
  for (int k = 0; k < W; ++k) z[4 + k] = w[k];
#pragma unroll
  for (int k = W + 7; k >= 2; --k) z[k] = (b & 8) ? z[k - 2] : z[k];
#pragma unroll
  for (int k = W + 7; k >= 1; --k) z[k] = (b & 4) ? z[k - 1] : z[k];
  const int sh = 8 * (b & 3);
  const int end = b + bytes;  // the run lies in [b, end) of the units from p - b on
#pragma unroll
  for (int u = 0; u <= W / 4; ++u) {
    const int o = 4 * W * lane + 16 * u;
    if (u == W / 4 && lane != 31) break;  // the next lane's first unit
    uint32_t x[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      x[k] = __funnelshift_l(z[4 * u + k + 3], z[4 * u + k + 4], sh);
    char* q = p - b + o;
    if (o >= b && o + 16 <= end) {
      *reinterpret_cast<uint4*>(q) = make_uint4(x[0], x[1], x[2], x[3]);
    } else if (o < end) {
      // [from, to) of the unit, in pieces that double up to 8 bytes and halve again
      const int from = o < b ? b : 0, to = end - o < 16 ? end - o : 16;
      int at = from;
#pragma unroll
      for (int d = 1; d <= 8; d *= 2)
        if ((at & d) && at + d <= to) {
          store_piece(q, x, at, d);
          at += d;
        }
#pragma unroll
      for (int d = 8; d >= 1; d /= 2)
        if (at + d <= to) {
          store_piece(q, x, at, d);
          at += d;
        }
    }
  }
}

__device__ __forceinline__ void ldg_v8(const void* p, uint32_t* w) {
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]),
                 "=r"(w[6]), "=r"(w[7])
               : "l"(p));
}
__device__ __forceinline__ void ldg_v4(const void* p, uint32_t* w) {
  asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
               : "l"(p));
}

__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// One chunk as it lies in memory: 8 words of BF16 pairs or 16 FP32 words; elements from n
// on are zero.
template <bool BF16>
struct Chunk {
  static constexpr int kWords = BF16 ? 8 : 16;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const void* base, int64_t off, int n, int grain) {
    const char* p = static_cast<const char*>(base) + off * (BF16 ? 2 : 4);
    if (n == kChunk && grain == 32) {
#pragma unroll
      for (int i = 0; i < kWords; i += 8) ldg_v8(p + 4 * i, w + i);
    } else if (n == kChunk && grain == 16) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4) ldg_v4(p + 4 * i, w + i);
    } else {
#pragma unroll
      for (int i = 0; i < kWords; ++i) w[i] = 0;
      if constexpr (BF16) {
        const uint16_t* q = reinterpret_cast<const uint16_t*>(p);
#pragma unroll
        for (int i = 0; i < kChunk; ++i)
          if (i < n) w[i >> 1] |= (uint32_t)q[i] << (16 * (i & 1));
      } else {
        const uint32_t* q = reinterpret_cast<const uint32_t*>(p);
#pragma unroll
        for (int i = 0; i < kChunk; ++i)
          if (i < n) w[i] = q[i];
      }
    }
  }
  // The same for a warp whose lanes hold consecutive chunks (`run` elements exist from lane
  // 0's on); smem: the warp's kStageBytes.  STAGED false: every grain is at least 16.
  template <bool STAGED>
  __device__ __forceinline__ void store_warp(void* base, int64_t off, int n, int64_t run,
                                             int grain, uint8_t* smem, int lane) const {
    if (!STAGED || grain >= 16) {
      store(base, off, n, grain);
      return;
    }
    constexpr int kElem = BF16 ? 2 : 4;
    char* p = static_cast<char*>(base) + (off - (int64_t)kChunk * lane) * kElem;
#pragma unroll
    for (int h = 0; h < kWords; h += 8)
      staged_store<8, 4 * kWords, kElem, 8>(p + 4 * h, (int)run * kElem - 4 * h, grain, smem,
                                            lane, w + h);
  }
  // From a row held in shared memory, 16-byte aligned (so n is a whole number of 16-byte
  // units).  Lanes are 32 or 64 bytes apart; rotating the order of a lane's units spreads
  // the eight lanes of an access over all banks.
  __device__ __forceinline__ void load_shared(const uint8_t* p, int n, int lane) {
    constexpr int kUnits = kWords / 4;
    const int rot = BF16 ? (lane >> 2) & 1 : (lane >> 1) & 3;
    uint4 u[kUnits];
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      const int at = (k + rot) & (kUnits - 1);
      u[k] = at * (kChunk / kUnits) < n ? *reinterpret_cast<const uint4*>(p + 16 * at)
                                        : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int d = 1; d < kUnits; d *= 2) {  // u[k] holds unit k + rot: rotate back
      uint4 r[kUnits];
#pragma unroll
      for (int k = 0; k < kUnits; ++k) {
        const uint4 a = u[k], b = u[(k - d) & (kUnits - 1)];
        r[k].x = (rot & d) ? b.x : a.x;
        r[k].y = (rot & d) ? b.y : a.y;
        r[k].z = (rot & d) ? b.z : a.z;
        r[k].w = (rot & d) ? b.w : a.w;
      }
#pragma unroll
      for (int k = 0; k < kUnits; ++k) u[k] = r[k];
    }
#pragma unroll
    for (int k = 0; k < kUnits; ++k) {
      w[4 * k] = u[k].x;
      w[4 * k + 1] = u[k].y;
      w[4 * k + 2] = u[k].z;
      w[4 * k + 3] = u[k].w;
    }
  }
  // The same for a chunk that starts at any element, by a whole warp whose lanes hold
  // consecutive chunks: aligned words, a lane's in an order rotated so that the 32 lanes of an
  // access hit all banks; the word that a chunk ends in is the next lane's first.  The words
  // around the row lie inside the stage; elements from n on come out as anything.
  __device__ __forceinline__ void load_shared_any(const uint8_t* p, int lane) {
    const uint32_t a = smem_addr(p);
    const uint32_t* q = reinterpret_cast<const uint32_t*>(p - (a & 3));
    const int rot = BF16 ? lane >> 2 : lane >> 1;  // modulo kWords
    uint32_t u[kWords];
#pragma unroll
    for (int k = 0; k < kWords; ++k) u[k] = q[(k + rot) & (kWords - 1)];
#pragma unroll
    for (int d = 1; d < kWords; d *= 2) {  // u[k] holds word k + rot: rotate back
      uint32_t r[kWords];
#pragma unroll
      for (int k = 0; k < kWords; ++k) r[k] = (rot & d) ? u[(k - d) & (kWords - 1)] : u[k];
#pragma unroll
      for (int k = 0; k < kWords; ++k) u[k] = r[k];
    }
    if constexpr (BF16) {
      uint32_t after = __shfl_down_sync(0xffffffffu, u[0], 1);
      if (lane == 31) after = q[kWords];
      const int sh = 8 * (int)(a & 2);
#pragma unroll
      for (int k = 0; k < kWords; ++k)
        w[k] = __funnelshift_r(u[k], k + 1 < kWords ? u[k + 1] : after, sh);
    } else {
#pragma unroll
      for (int k = 0; k < kWords; ++k) w[k] = u[k];
    }
  }
  // Elements from n on become zero.
  __device__ __forceinline__ void cut(int n) {
    if (n >= kChunk) return;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      if (i < n) continue;
      if constexpr (BF16) w[i >> 1] &= (i & 1) ? 0x0000ffffu : 0xffff0000u;
      else w[i] = 0;
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (BF16) return (i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
    else return __uint_as_float(w[i]);
  }
  // Round 16 values into the chunk (nearest even).
  __device__ __forceinline__ void set(const float* v) {
    if constexpr (BF16) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = bf16x2_bits(v[2 * i], v[2 * i + 1]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = __float_as_uint(v[i]);
    }
  }
  __device__ __forceinline__ void store(void* base, int64_t off, int n, int grain) const {
    char* p = static_cast<char*>(base) + off * (BF16 ? 2 : 4);
    if (n == kChunk && grain == 32) {
#pragma unroll
      for (int i = 0; i < kWords; i += 8) stg_v8(p + 4 * i, w + i);
    } else if (n == kChunk && grain == 16) {
#pragma unroll
      for (int i = 0; i < kWords; i += 4)
        *reinterpret_cast<uint4*>(p + 4 * i) = make_uint4(w[i], w[i + 1], w[i + 2], w[i + 3]);
    } else if constexpr (BF16) {
      uint16_t* q = reinterpret_cast<uint16_t*>(p);
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        if (i < n) q[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    } else {
      uint32_t* q = reinterpret_cast<uint32_t*>(p);
#pragma unroll
      for (int i = 0; i < kChunk; ++i)
        if (i < n) q[i] = w[i];
    }
  }
};

// A chunk's load by a warp whose lanes hold consecutive chunks, in two steps: issue() for
// every tensor first, then settle() one after the other.  STAGED false: every grain is at
// least 16, and settle has nothing to do.
template <bool BF16, bool STAGED>
struct ChunkLoad {
  Chunk<BF16> c;
  StagedLoad<8, 4 * Chunk<BF16>::kWords, BF16 ? 2 : 4> raw[STAGED ? Chunk<BF16>::kWords / 8 : 1];

  __device__ __forceinline__ void issue(const void* base, int64_t off, int n, int64_t run,
                                        int grain, int lane) {
    if (!STAGED || grain >= 16) {
      c.load(base, off, n, grain);
      return;
    }
    constexpr int kElem = BF16 ? 2 : 4;
    const char* p = static_cast<const char*>(base) + (off - (int64_t)kChunk * lane) * kElem;
#pragma unroll
    for (int h = 0; h < Chunk<BF16>::kWords / 8; ++h)
      raw[h].issue(p + 32 * h, (int)run * kElem - 32 * h, grain, lane);
  }
  __device__ __forceinline__ const Chunk<BF16>& settle(int grain, uint8_t* smem, int lane) {
    if constexpr (STAGED) {
      if (grain < 16) {
#pragma unroll
        for (int h = 0; h < Chunk<BF16>::kWords / 8; ++h)
          raw[h].settle(grain, smem, lane, c.w + 8 * h);
      }
    }
    return c;
  }
};

// The 16 FP32 values of a chunk of a BF16 or FP32 vector (type known at run time).
__device__ __forceinline__ void load_vector16(const void* base, bool bf16, int64_t off, int n,
                                              int grain, float* v) {
  if (bf16) {
    Chunk<true> c;
    c.load(base, off, n, grain);
#pragma unroll
    for (int i = 0; i < kChunk; ++i) v[i] = c.get(i);
  } else {
    Chunk<false> c;
    c.load(base, off, n, grain);
#pragma unroll
    for (int i = 0; i < kChunk; ++i) v[i] = c.get(i);
  }
}

// Contiguous bytes to shared memory, completing on `bar` (16-byte aligned addresses, size a
// multiple of 16).
__device__ __forceinline__ void bulk_copy_in(void* dst, const void* src, uint32_t bytes,
                                             uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(smem_addr(bar))
      : "memory");
}

// Elements from column c on of a row of `cols`, for a warp (at most its 32 chunks).
__device__ __forceinline__ int64_t warp_run(int64_t c, int64_t cols) {
  const int64_t left = cols - c;
  return left < 0 ? 0 : (left < 32 * kChunk ? left : 32 * kChunk);
}

// Elements of the chunk that starts at column c of a row of `cols` (0 past its end).
__device__ __forceinline__ int chunk_len(int64_t c, int64_t cols) {
  const int64_t left = cols - c;
  return left >= kChunk ? kChunk : (left > 0 ? (int)left : 0);
}

}  // namespace nvfp4
