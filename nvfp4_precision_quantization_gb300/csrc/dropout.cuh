// dropout.cuh -- a dropout mask that is never stored: element i's bit follows from the call's
// seed and offset, wherever and however often it is asked for.
//
// Philox4x32 with ten rounds (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy as
// 1, 2, 3", 2011): a round multiplies two of the four counter words by constants, and the
// halves of the 64-bit products, mixed with the key, are the next words.  A block of counter
// (i / 8, offset) gives element i its 16 bits, half i % 2 of word i % 8 / 2: eight elements a
// block is what keeps the generator (18 products of 32 x 32 -> 64 bits and as many exclusive ors a block)
// below the memory time of the passes that it is part of; with 32 bits an element it would cost
// twice that.  An element is dropped where its bits are below threshold = round(p
// 2^16), and what is kept is scaled by 1 / (1 - threshold 2^-16): unbiased for the rounded p.
#pragma once

#include "internal.h"
#include "row_io.cuh"

namespace nvfp4 {

struct PhiloxBlock {
  uint32_t w[4];
};

// A call's mask inside a kernel.  The round keys are read from the kernel's arguments.
struct Dropper {
  const DropMask& m;
  uint32_t below;  // kept: 16 bits greater than `below` = threshold - 1
  bool on;         // false: everything is kept as it is
  // The first round's second product, of a counter word that is the call's offset, is the same
  // for all blocks, and so is the second round's first one where the blocks' upper words are 0.
  uint32_t first0, first1, first2;  // words 0, 1 of the second round's counter, less block's upper
                                    // word; what mixes into word 2
  uint32_t second_high, second_low;

  __device__ __forceinline__ explicit Dropper(const DropMask& mask)
      : m(mask), below(mask.threshold - 1), on(mask.threshold != 0) {
    uint64_t offset = m.offset;
    if (on && m.offset_add != nullptr) offset += __ldg(m.offset_add);
    const uint64_t b = (uint64_t)(uint32_t)offset * kMul1;
    first0 = (uint32_t)(b >> 32) ^ m.key0[0];
    first1 = (uint32_t)b;
    first2 = (uint32_t)(offset >> 32) ^ m.key1[0];
    const uint64_t a = (uint64_t)first0 * kMul0;
    second_high = (uint32_t)(a >> 32) ^ m.key1[1];
    second_low = (uint32_t)a;
  }
  static constexpr uint32_t kMul0 = 0xD2511F53u, kMul1 = 0xCD9E8D57u;

  __device__ __forceinline__ PhiloxBlock philox(uint64_t block) const {
    const uint32_t upper = (uint32_t)(block >> 32);
    uint64_t a = (uint64_t)(uint32_t)block * kMul0;
    // after round 0: (first0 ^ upper, first1, high(a) ^ first2, low(a))
    uint64_t b = (uint64_t)((uint32_t)(a >> 32) ^ first2) * kMul1;
    uint32_t high = second_high, low = second_low;
    if (upper != 0) {  // more than 2^35 elements
      const uint64_t c = (uint64_t)(first0 ^ upper) * kMul0;
      high = (uint32_t)(c >> 32) ^ m.key1[1];
      low = (uint32_t)c;
    }
    uint32_t c0 = (uint32_t)(b >> 32) ^ first1 ^ m.key0[1], c1 = (uint32_t)b;
    uint32_t c2 = high ^ (uint32_t)a, c3 = low;
#pragma unroll
    for (int r = 2; r < 10; ++r) {
      a = (uint64_t)c0 * kMul0, b = (uint64_t)c2 * kMul1;
      c0 = (uint32_t)(b >> 32) ^ c1 ^ m.key0[r];
      c2 = (uint32_t)(a >> 32) ^ c3 ^ m.key1[r];
      c1 = (uint32_t)b;
      c3 = (uint32_t)a;
    }
    return {{c0, c1, c2, c3}};
  }
  // The bits of elements e .. e + 15 (e >= 0), two in a word.
  __device__ __forceinline__ void words(int64_t e, uint32_t (&z)[kChunk / 2]) const {
    const uint64_t block = (uint64_t)e >> 3;
    const int shift = (int)(e & 7);  // rows of no multiple of 8 start inside a block
    const PhiloxBlock a = philox(block), b = philox(block + 1);
#pragma unroll
    for (int i = 0; i < 4; ++i) z[i] = a.w[i], z[4 + i] = b.w[i];
    if (shift == 0) return;
    const PhiloxBlock c = philox(block + 2);
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
  // infinity too), plus r's (where there are any): a comparison and an FMA an element.
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
    const float scale = m.scale;
#pragma unroll
    for (int i = 0; i < kChunk; ++i) {
      const float b = r != nullptr ? r->get(i) : 0.0f;
      const bool keep = (i & 1) ? z[i / 2] > high : (z[i / 2] & 0xffffu) > below;
      float o = b;
      if (keep) o = __fmaf_rn(v[i], scale, b);
      v[i] = o;
    }
  }
};

}  // namespace nvfp4
