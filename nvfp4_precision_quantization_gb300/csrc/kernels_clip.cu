// kernels_clip.cu -- the global 2-norm of a list of gradients, and clipping by it.
//
//   norm = sqrt(sum g^2),  out = g min(1, max_norm / (norm + 1e-6))
//
// Bound by memory: the norm must be known before the first scaled value, so the list is
// read twice and written once.  The list travels in the kernels' arguments (no device
// table to keep or to copy) and is cut into pieces of kPiece values that a persistent
// grid walks, the second pass backwards, from what the first read last (worth 1 to 2 %:
// holding the tail in L2 with evict-last loads, giving a piece to the same CTA in both
// passes and streaming stores added nothing measurable).  Each CTA of the first pass leaves one
// FP64 partial sum; each CTA of the second adds them all, in the same order, instead of
// waiting for a kernel between the two.
//
// Measured: 973 M BF16 values into a second buffer 900 us: 280 us for the first pass (6.95
// TB/s) and 597 us for the second (6.45 TB/s) when each is run cold.
#include <algorithm>

#include "internal.h"
#include "row_io.cuh"

namespace nvfp4 {
namespace {

constexpr int kClipThreads = 512;
constexpr int kPiece = kClipThreads * kChunk * 2;  // values of a piece: two chunks a thread
// Tensors of one launch: the arguments of a short list are copied faster.
constexpr int kShortList = 64, kListCapacity = 512;
constexpr int kClipMaxCtas = 1024;                 // partial sums per launch

struct ListEntry {
  const void* data;
  void* out;
  int64_t n;
  int64_t first;  // the tensor's first piece
};
template <int CAP>
struct ListArgs {
  int count;
  int64_t pieces;
  uint32_t bf16[CAP / 32];
  ListEntry e[CAP];
};

// The entry that holds piece p: the last one whose first piece is at most p (empty
// tensors have no piece and share their first with the next entry).
template <int CAP>
__device__ __forceinline__ int find_entry(const ListArgs<CAP>& a, int64_t p) {
  int lo = 0, hi = a.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.e[mid].first <= p) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}
template <int CAP>
__device__ __forceinline__ bool entry_bf16(const ListArgs<CAP>& a, int i) {
  return (a.bf16[i >> 5] >> (i & 31)) & 1u;
}
__device__ __forceinline__ int pointer_grain(const void* p) {
  const uintptr_t u = reinterpret_cast<uintptr_t>(p);
  return (u & 31) == 0 ? 32 : ((u & 15) == 0 ? 16 : 0);
}

template <bool BF16>
__device__ __forceinline__ float piece_squares(const void* data, int64_t at, int64_t n) {
  const int grain = pointer_grain(data);
  Chunk<BF16> c[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int64_t off = at + (k * kClipThreads + (int)threadIdx.x) * kChunk;
    c[k].load(data, off, chunk_len(off, n), grain);
  }
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < kChunk; ++i) s[i & 3] = __fmaf_rn(c[k].get(i), c[k].get(i), s[i & 3]);
  return __fadd_rn(__fadd_rn(s[0], s[1]), __fadd_rn(s[2], s[3]));
}

template <bool BF16>
__device__ __forceinline__ void piece_scale(const void* data, void* out, int64_t at, int64_t n,
                                            float coef) {
  const int grain = pointer_grain(data), grain_out = pointer_grain(out);
  Chunk<BF16> c[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int64_t off = at + (k * kClipThreads + (int)threadIdx.x) * kChunk;
    c[k].load(data, off, chunk_len(off, n), grain);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int64_t off = at + (k * kClipThreads + (int)threadIdx.x) * kChunk;
    float v[kChunk];
#pragma unroll
    for (int i = 0; i < kChunk; ++i) v[i] = __fmul_rn(c[k].get(i), coef);
    c[k].set(v);
    c[k].store(out, off, chunk_len(off, n), grain_out);
  }
}

// Sum of one double per thread over the CTA, in a fixed order; valid in thread 0.
__device__ __forceinline__ double block_sum(double v, double* s) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  if (threadIdx.x == 0)
    for (int i = 1; i < (int)blockDim.x / 32; ++i) v += s[i];
  return v;
}

template <int CAP>
__global__ void __launch_bounds__(kClipThreads)
    k_square_sum(const __grid_constant__ ListArgs<CAP> a, double* part) {
  __shared__ double s[kClipThreads / 32];
  double sum = 0.0;
  for (int64_t p = blockIdx.x; p < a.pieces; p += gridDim.x) {
    const int i = find_entry(a, p);
    const int64_t at = (p - a.e[i].first) * kPiece;
    sum += (double)(entry_bf16(a, i) ? piece_squares<true>(a.e[i].data, at, a.e[i].n)
                                     : piece_squares<false>(a.e[i].data, at, a.e[i].n));
  }
  pdl_launch_dependents();
  sum = block_sum(sum, s);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// The norm from the partial sums, in thread 0 (the same bits in every CTA).
__device__ __forceinline__ float norm_of(const double* part, int parts, double* s) {
  double sum = 0.0;
  for (int i = threadIdx.x; i < parts; i += kClipThreads) sum += part[i];
  return (float)sqrt(block_sum(sum, s));
}

__global__ void __launch_bounds__(kClipThreads)
    k_list_norm(const double* part, int parts, float* norm) {
  __shared__ double s[kClipThreads / 32];
  pdl_wait();
  const float v = norm_of(part, parts, s);
  if (threadIdx.x == 0) *norm = v;
}

template <int CAP>
__global__ void __launch_bounds__(kClipThreads)
    k_clip(const __grid_constant__ ListArgs<CAP> a, const double* part, int parts, float max_norm,
           float* norm) {
  __shared__ double s[kClipThreads / 32];
  __shared__ float s_coef;
  pdl_wait();
  const float v = norm_of(part, parts, s);
  if (threadIdx.x == 0) {
    const float c = __fdiv_rn(max_norm, __fadd_rn(v, 1e-6f));
    s_coef = c >= 1.0f ? 1.0f : c;  // NaN stays NaN
    if (blockIdx.x == 0 && norm != nullptr) *norm = v;
  }
  __syncthreads();
  const float coef = s_coef;
  for (int64_t p = a.pieces - 1 - blockIdx.x; p >= 0; p -= gridDim.x) {
    const int i = find_entry(a, p);
    // in place and nothing to scale
    if (coef == 1.0f && a.e[i].out == a.e[i].data) continue;
    const int64_t at = (p - a.e[i].first) * kPiece;
    if (entry_bf16(a, i)) piece_scale<true>(a.e[i].data, a.e[i].out, at, a.e[i].n, coef);
    else piece_scale<false>(a.e[i].data, a.e[i].out, at, a.e[i].n, coef);
  }
}

template <int CAP>
int64_t fill_list(const TensorEntry* t, int count, ListArgs<CAP>* a) {
  a->count = count;
  int64_t first = 0;
  for (int i = 0; i < count; ++i) {
    a->e[i] = {t[i].data, t[i].out, t[i].n, first};
    if (t[i].bf16) a->bf16[i >> 5] |= 1u << (i & 31);
    first += (t[i].n + kPiece - 1) / kPiece;
  }
  return a->pieces = first;
}

template <int CAP>
cudaError_t run_clip(const TensorEntry* t, int count, bool clip, float max_norm, float* norm,
                     double* part, const DeviceInfo& dev, cudaStream_t stream) {
  const int max_grid = std::min(kClipMaxCtas, 2 * dev.num_sms);
  int parts = 0;
  for (int i = 0; i < count; i += CAP) {
    ListArgs<CAP> a{};
    const int64_t pieces = fill_list(t + i, std::min(CAP, count - i), &a);
    if (pieces == 0) continue;
    const int grid = (int)std::min<int64_t>(pieces, max_grid);
    k_square_sum<<<grid, kClipThreads, 0, stream>>>(a, part + parts);
    parts += grid;
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  bool written = false;
  for (int i = (count - 1) / CAP * CAP; clip && i >= 0; i -= CAP) {
    ListArgs<CAP> a{};
    const int64_t pieces = fill_list(t + i, std::min(CAP, count - i), &a);
    if (pieces == 0) continue;
    const int grid = (int)std::min<int64_t>(pieces, max_grid);
    float* out = written ? nullptr : norm;
    // A dependent launch saves 1 us where every CTA has one piece; on longer lists it
    // disturbs the reuse of L2 (20 M values: 37 us plainly launched, 40 dependent).
    cudaError_t e;
    if (pieces <= max_grid) {
      e = launch_after(k_clip<CAP>, (unsigned)grid, kClipThreads, stream, a, (const double*)part,
                       parts, max_norm, out);
    } else {
      k_clip<CAP><<<grid, kClipThreads, 0, stream>>>(a, part, parts, max_norm, out);
      e = cudaGetLastError();
    }
    if (e != cudaSuccess) return e;
    written = true;
  }
  if (written) return cudaSuccess;
  return launch_after(k_list_norm, 1, kClipThreads, stream, (const double*)part, parts, norm);
}

}  // namespace

int64_t clip_workspace() { return (int64_t)kClipMaxCtas * kClipMaxLaunches * sizeof(double); }
int64_t clip_capacity() { return (int64_t)kListCapacity * kClipMaxLaunches; }

cudaError_t launch_clip(const TensorEntry* t, int count, bool clip, float max_norm, float* norm,
                        void* workspace, const DeviceInfo& dev, cudaStream_t stream) {
  double* part = static_cast<double*>(workspace);
  return count <= kShortList
             ? run_clip<kShortList>(t, count, clip, max_norm, norm, part, dev, stream)
             : run_clip<kListCapacity>(t, count, clip, max_norm, norm, part, dev, stream);
}

}  // namespace nvfp4
