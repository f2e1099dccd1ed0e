// dropout.cuh -- a dropout mask that is never stored: element i's bit follows from the call's
// seed and offset, wherever and however often it is asked for.
//
// Philox4x32 with ten rounds (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as
// 1, 2, 3", 2011): a round multiplies two of the four counter words by constants, and the
// halves of the 64-bit products, mixed with the key, are the next words.  A block of counter
// (i / 8, offset) gives element i its 16 bits, half i % 2 of word i % 8 / 2: eight elements a
// block is what keeps the generator (42 instructions a block, 20 of them 32 x 32 -> 64 bit
// products) below the memory time of the passes that it is part of; with 32 bits an element it
// would cost twice that.  An element is dropped where its bits are below threshold = round(p
// 2^16), and what is kept is scaled by 1 / (1 - threshold 2^-16): unbiased for the rounded p.
#pragma once

#include "internal.h"
#include "row_io.cuh"

namespace nvfp4 {

struct PhiloxBlock {
  uint32_t w[4];
};
__device__ __forceinline__ PhiloxBlock philox(uint64_t block, uint64_t offset, uint32_t k0,
                                              uint32_t k1) {
  uint32_t c0 = (uint32_t)block, c1 = (uint32_t)(block >> 32);
  uint32_t c2 = (uint32_t)offset, c3 = (uint32_t)(offset >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t a = (uint64_t)c0 * 0xD2511F53u, b = (uint64_t)c2 * 0xCD9E8D57u;
    c0 = (uint32_t)(b >> 32) ^ c1 ^ k0;
    c2 = (uint32_t)(a >> 32) ^ c3 ^ k1;
    c1 = (uint32_t)b;
    c3 = (uint32_t)a;
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return {{c0, c1, c2, c3}};
}

// A call's mask inside a kernel.
struct Dropper {
  uint32_t k0, k1, below;  // kept: 16 bits greater than `below` = threshold - 1
  uint64_t offset;
  float scale;
  bool on;  // false: everything is kept as it is
  __device__ __forceinline__ explicit Dropper(const DropMask& m)
      : k0(m.key0), k1(m.key1), below(m.threshold - 1), offset(m.offset), scale(m.scale),
        on(m.threshold != 0) {
    if (on && m.offset_add != nullptr) offset += __ldg(m.offset_add);
  }
  // The bits of elements e .. e + 15 (e >= 0), two in a word.
  __device__ __forceinline__ void words(int64_t e, uint32_t (&z)[kChunk / 2]) const {
    const uint64_t block = (uint64_t)e >> 3;
    const int shift = (int)(e & 7);  // rows of no multiple of 8 start inside a block
    const PhiloxBlock a = philox(block, offset, k0, k1), b = philox(block + 1, offset, k0, k1);
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = a.w[i], z[4 + i] = b.w[i];
    if (shift == 0) return;
    const PhiloxBlock c = philox(block + 2, offset, k0, k1);
    uint32_t x[12];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = z[i];
#pragma unroll
    for (int i = 0; i < 4; ++i) x[8 + i] = c.w[i];
#pragma unroll
    for (int i = 0; i < 10; ++i) x[i] = (shift & 4) ? x[i + 2] : x[i];
#pragma unroll
    for (int i = 0; i < 9; ++i) x[i] = (shift & 2) ? x[i + 1] : x[i];
#pragma unroll
    for (int i = 0; i < 8; ++i) z[i] = __funnelshift_r(x[i], x[i + 1], 16 * (shift & 1));
  }
  // v[0 .. 16), the elements from e on, scaled where kept and zero where dropped (a NaN or an
  // infinity too), plus r's (where there are any): one FMA and one selection an element.
  template <bool BF16>
  __device__ __forceinline__ void apply(int64_t e, float* v, const Chunk<BF16>* r) const {
    if (!on) {
      if (r == nullptr) return;
#pragma unroll
      for (int i = 0; i < kChunk; i += 2) {
        const Pair s = pair_add({v[i], v[i + 1]}, {r->get(i), r->get(i + 1)});
        v[i] = s.x;
        v[i + 1] = s.y;
      }
      return;
    }
    uint32_t z[kChunk / 2];
    words(e, z);
    const uint32_t high = (below << 16) | 0xffffu;
#pragma unroll
    for (int i = 0; i < kChunk; i += 2) {
      const Pair b = r != nullptr ? Pair{r->get(i), r->get(i + 1)} : Pair{0.0f, 0.0f};
      const Pair s = pair_fma({v[i], v[i + 1]}, {scale, scale}, b);
      v[i] = (z[i / 2] & 0xffffu) > below ? s.x : b.x;
      v[i + 1] = z[i / 2] > high ? s.y : b.y;
    }
  }
};

}  // namespace nvfp4
