// api_layer.cu -- the C ABI of the layer operators (norm, bias and activation, gradient
// clipping): argument checks and launches, by the conventions of api.cu.
#include <memory>

#include "api_common.h"

using namespace nvfp4;

namespace {

bool aligned(const void* p, size_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }

int64_t elem_bytes(int32_t dtype) { return dtype == NVFP4_IN_BF16 ? 2 : 4; }

// Every pointer that is given must be aligned to its element.
nvfp4_status check_elems(std::initializer_list<const void*> ptrs, int32_t dtype) {
  for (const void* p : ptrs)
    if (!aligned(p, elem_bytes(dtype)))
      return fail(NVFP4_ERR_INVALID, "a tensor is not aligned to its element size");
  return NVFP4_OK;
}

nvfp4_status check_norm(int32_t in_dtype, int32_t weight_dtype, const void* weight, int64_t rows,
                        int64_t cols) {
  nvfp4_status st;
  if (!valid_in_dtype(in_dtype)) return fail(NVFP4_ERR_INVALID, "unknown in_dtype");
  if (!valid_in_dtype(weight_dtype)) return fail(NVFP4_ERR_INVALID, "unknown weight_dtype");
  if ((st = check_sizes(rows, cols)) != NVFP4_OK) return st;
  if (cols > NVFP4_RMSNORM_MAX_COLS)
    return fail(NVFP4_ERR_UNSUPPORTED, "cols exceeds NVFP4_RMSNORM_MAX_COLS");
  if (weight == nullptr && rows * cols > 0) return fail(NVFP4_ERR_INVALID, "weight is NULL");
  return check_elems({weight}, weight_dtype);
}

nvfp4_status check_workspace(const void* workspace, uint64_t have, uint64_t need) {
  if (need == 0) return NVFP4_OK;
  if (workspace == nullptr || !aligned(workspace, 16))
    return fail(NVFP4_ERR_INVALID, "workspace must be non-NULL and 16-byte aligned");
  if (have < need)
    return fail(NVFP4_ERR_INVALID,
                "workspace of " + std::to_string(have) + " bytes, " + std::to_string(need) +
                    " needed");
  return NVFP4_OK;
}

// Whether out shares bytes with in without starting where it starts (an element written
// before another thread reads it).
bool shifted(const void* out, const void* in, uint64_t bytes) {
  return out != in && bytes_overlap(out, bytes, in, bytes);
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_add_rmsnorm(const void* x, const void* residual, int32_t in_dtype,
                               const void* weight, int32_t weight_dtype, int64_t rows,
                               int64_t cols, float eps, void* h, void* y, float* rstd,
                               const nvfp4_fp8_out* fp8, const nvfp4_config* cfg,
                               const nvfp4_out* row, nvfp4_stream_t stream) {
  nvfp4_status st;
  if ((st = check_norm(in_dtype, weight_dtype, weight, rows, cols)) != NVFP4_OK) return st;
  if ((st = check_elems({x, residual, h, y}, in_dtype)) != NVFP4_OK) return st;
  if ((st = check_elems({rstd}, NVFP4_IN_FP32)) != NVFP4_OK) return st;
  if (!(eps >= 0.0f)) return fail(NVFP4_ERR_INVALID, "eps must be >= 0");
  if (x == nullptr && rows * cols > 0) return fail(NVFP4_ERR_INVALID, "x is NULL");
  if (h != nullptr && residual == nullptr)
    return fail(NVFP4_ERR_INVALID, "h is the sum with a residual: residual is NULL");
  if (rows * cols > 0 && y == nullptr && fp8 == nullptr && row == nullptr)
    return fail(NVFP4_ERR_INVALID, "no output: y, fp8 and row are NULL");
  if (fp8 != nullptr && row != nullptr)
    return fail(NVFP4_ERR_UNSUPPORTED, "fp8 and row outputs in one call");
  const uint64_t bytes = (uint64_t)(rows * cols * elem_bytes(in_dtype));
  if (bytes_overlap(h, bytes, y, bytes)) return fail(NVFP4_ERR_INVALID, "h overlaps y");
  for (const void* in : {x, residual})
    if (shifted(h, in, bytes) || shifted(y, in, bytes))
      return fail(NVFP4_ERR_INVALID, "h or y overlaps x or residual without being it");
  NormArgs n{};
  if (fp8 != nullptr) {
    if (fp8->block != 0 && fp8->block != 128)
      return fail(NVFP4_ERR_INVALID, "fp8->block must be 0 or 128");
    if (fp8->codes == nullptr && rows * cols > 0)
      return fail(NVFP4_ERR_INVALID, "fp8->codes is NULL");
    const int64_t scales = fp8->block ? rows * ((cols + 127) / 128) : rows;
    if (fp8->scale == nullptr && scales > 0)
      return fail(NVFP4_ERR_INVALID, "fp8->scale is NULL");
    if ((st = check_elems({fp8->scale}, NVFP4_IN_FP32)) != NVFP4_OK) return st;
    n.q8 = fp8->codes;
    n.q8_scale = fp8->scale;
    n.q8_block = fp8->block;
    // empty rows still have their scale: any non-NULL codes pointer, never written
    if (n.q8 == nullptr) n.q8 = reinterpret_cast<uint8_t*>(n.q8_scale);
  }
  if (row != nullptr) {
    if ((st = check_config(cfg)) != NVFP4_OK) return st;
    if (cfg->block_2d)
      return fail(NVFP4_ERR_UNSUPPORTED, "16x16 blocks span rows: quantize y instead");
    const bool per_tensor = cfg->mode == NVFP4_PER_TENSOR;
    if ((st = check_out(row, "row", rows, cols, per_tensor ? 1 : rows)) != NVFP4_OK) return st;
    if (per_tensor && row->amax_in == nullptr)
      return fail(NVFP4_ERR_UNSUPPORTED,
                  "NVFP4_PER_TENSOR needs row->amax_in (the tensor's amax is not known in one "
                  "pass): give it, or use NVFP4_ROW_SCALED");
    n.codes = row->codes;
    n.scales = row->scales;
    n.amax = row->amax;
    n.amax_in = row->amax_in;
    n.amax_per_tensor = per_tensor;
    n.four_over_six = cfg->four_over_six != 0;
    n.bound = cfg->bound;
  }
  if (rows == 0) return NVFP4_OK;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != NVFP4_OK) return st;
  n.x = x;
  n.residual = residual;
  n.in = in_dtype == NVFP4_IN_BF16 ? InType::BF16 : InType::FP32;
  n.weight = weight;
  n.weight_bf16 = weight_dtype == NVFP4_IN_BF16;
  n.rows = rows;
  n.cols = cols;
  n.eps = eps;
  n.h = h;
  n.y = y;
  n.rstd = rstd;
  cudaError_t e = launch_add_rmsnorm(n, dev, stream);
  return e == cudaSuccess ? NVFP4_OK : cuda_fail(e, "norm launch");
}

nvfp4_status nvfp4_add_rmsnorm_backward_workspace_size(int64_t rows, int64_t cols,
                                                       uint64_t* bytes) {
  if (bytes == nullptr) return fail(NVFP4_ERR_INVALID, "bytes is NULL");
  nvfp4_status st = check_sizes(rows, cols);
  if (st != NVFP4_OK) return st;
  *bytes = (uint64_t)add_rmsnorm_backward_workspace(rows, cols);
  return NVFP4_OK;
}

nvfp4_status nvfp4_add_rmsnorm_backward(const void* dy, const void* h, const void* dh,
                                        int32_t in_dtype, const void* weight,
                                        int32_t weight_dtype, const float* rstd, int64_t rows,
                                        int64_t cols, void* dx, float* dweight, void* workspace,
                                        uint64_t workspace_bytes, nvfp4_stream_t stream) {
  nvfp4_status st;
  if ((st = check_norm(in_dtype, weight_dtype, weight, rows, cols)) != NVFP4_OK) return st;
  if ((st = check_elems({dy, h, dh, dx}, in_dtype)) != NVFP4_OK) return st;
  if ((st = check_elems({rstd, dweight}, NVFP4_IN_FP32)) != NVFP4_OK) return st;
  if (rows * cols > 0 && (dy == nullptr || h == nullptr || rstd == nullptr || dx == nullptr))
    return fail(NVFP4_ERR_INVALID, "dy, h, rstd and dx must be non-NULL");
  const uint64_t bytes = (uint64_t)(rows * cols * elem_bytes(in_dtype));
  for (const void* in : {dy, h, dh})
    if (shifted(dx, in, bytes))
      return fail(NVFP4_ERR_INVALID, "dx overlaps an input without being it");
  if (dweight != nullptr &&
      (st = check_workspace(workspace, workspace_bytes,
                            (uint64_t)add_rmsnorm_backward_workspace(rows, cols))) != NVFP4_OK)
    return st;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != NVFP4_OK) return st;
  NormBackwardArgs n{};
  n.dy = dy;
  n.h = h;
  n.dh = dh;
  n.in = in_dtype == NVFP4_IN_BF16 ? InType::BF16 : InType::FP32;
  n.weight = weight;
  n.weight_bf16 = weight_dtype == NVFP4_IN_BF16;
  n.rstd = rstd;
  n.rows = rows;
  n.cols = cols;
  n.dx = dx;
  n.dweight = dweight;
  n.workspace = workspace;
  cudaError_t e = launch_add_rmsnorm_backward(n, dev, stream);
  return e == cudaSuccess ? NVFP4_OK : cuda_fail(e, "norm backward launch");
}

nvfp4_status nvfp4_bias_act_backward_workspace_size(int64_t rows, int64_t cols,
                                                    uint64_t* bytes) {
  if (bytes == nullptr) return fail(NVFP4_ERR_INVALID, "bytes is NULL");
  nvfp4_status st = check_sizes(rows, cols);
  if (st != NVFP4_OK) return st;
  *bytes = rows * cols > 0 ? (uint64_t)bias_act_backward_workspace(rows, cols) : 0;
  return NVFP4_OK;
}

nvfp4_status nvfp4_bias_act_backward(const void* dd, const void* z, int32_t dtype, int32_t act,
                                     int64_t rows, int64_t cols, void* dz, float* dbias,
                                     float* row_amax, float* col_amax, void* workspace,
                                     uint64_t workspace_bytes, nvfp4_stream_t stream) {
  nvfp4_status st;
  if (!valid_in_dtype(dtype)) return fail(NVFP4_ERR_INVALID, "unknown dtype");
  if (!valid_activation(act)) return fail(NVFP4_ERR_INVALID, "unknown activation");
  if ((st = check_sizes(rows, cols)) != NVFP4_OK) return st;
  if ((st = check_elems({dd, z, dz}, dtype)) != NVFP4_OK) return st;
  if ((st = check_elems({dbias, row_amax, col_amax}, NVFP4_IN_FP32)) != NVFP4_OK) return st;
  if (rows * cols > 0) {
    if (dd == nullptr || dz == nullptr)
      return fail(NVFP4_ERR_INVALID, "dd and dz must be non-NULL");
    if (z == nullptr && act != NVFP4_ACT_NONE)
      return fail(NVFP4_ERR_INVALID, "z is NULL: the activation's gradient needs it");
  }
  const uint64_t bytes = (uint64_t)(rows * cols * elem_bytes(dtype));
  if (shifted(dz, dd, bytes) || (act != NVFP4_ACT_NONE && shifted(dz, z, bytes)))
    return fail(NVFP4_ERR_INVALID, "dz overlaps an input without being it");
  if (rows * cols > 0 && (dbias || row_amax || col_amax) &&
      (st = check_workspace(workspace, workspace_bytes,
                            (uint64_t)bias_act_backward_workspace(rows, cols))) != NVFP4_OK)
    return st;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != NVFP4_OK) return st;
  ActBackwardArgs a{};
  a.dd = dd;
  a.z = z;
  a.in = dtype == NVFP4_IN_BF16 ? InType::BF16 : InType::FP32;
  a.act = act;
  a.rows = rows;
  a.cols = cols;
  a.dz = dz;
  a.dbias = dbias;
  a.row_amax = row_amax;
  a.col_amax = col_amax;
  a.workspace = workspace;
  cudaError_t e = launch_bias_act_backward(a, dev, stream);
  return e == cudaSuccess ? NVFP4_OK : cuda_fail(e, "activation backward launch");
}

nvfp4_status nvfp4_clip_grad_norm_workspace_size(uint64_t* bytes) {
  if (bytes == nullptr) return fail(NVFP4_ERR_INVALID, "bytes is NULL");
  *bytes = (uint64_t)clip_workspace();
  return NVFP4_OK;
}

namespace {
nvfp4_status clip_impl(const nvfp4_tensor* tensors, int32_t count, bool clip, float max_norm,
                       float* norm, void* workspace, uint64_t workspace_bytes,
                       nvfp4_stream_t stream) {
  nvfp4_status st;
  if (count < 0) return fail(NVFP4_ERR_INVALID, "count must be >= 0");
  if (count > clip_capacity())
    return fail(NVFP4_ERR_UNSUPPORTED,
                "more than " + std::to_string(clip_capacity()) + " tensors in one list");
  if (tensors == nullptr && count > 0) return fail(NVFP4_ERR_INVALID, "tensors is NULL");
  if (clip && !(max_norm >= 0.0f)) return fail(NVFP4_ERR_INVALID, "max_norm must be >= 0");
  if (norm == nullptr || !aligned(norm, 4))
    return fail(NVFP4_ERR_INVALID, "norm must be non-NULL and 4-byte aligned");
  std::unique_ptr<TensorEntry[]> list(new (std::nothrow) TensorEntry[count > 0 ? count : 1]);
  if (!list) return fail(NVFP4_ERR_INVALID, "out of host memory");
  for (int32_t i = 0; i < count; ++i) {
    const nvfp4_tensor& t = tensors[i];
    const char* bad = nullptr;
    if (!valid_in_dtype(t.dtype)) bad = "unknown dtype";
    else if (t.n < 0 || t.n >= (1LL << 48)) bad = "n out of range";
    else if (t.n > 0 && (t.data == nullptr || (clip && t.out == nullptr)))
      bad = "data or out is NULL";
    else if (!aligned(t.data, elem_bytes(t.dtype)) ||
             (clip && !aligned(t.out, elem_bytes(t.dtype))))
      bad = "not aligned to its element size";
    else if (clip && shifted(t.out, t.data, (uint64_t)(t.n * elem_bytes(t.dtype))))
      bad = "out overlaps data without being it";
    if (bad) return fail(NVFP4_ERR_INVALID, "tensor " + std::to_string(i) + ": " + bad);
    list[i] = {t.data, t.out, t.n, t.dtype == NVFP4_IN_BF16};
  }
  if ((st = check_workspace(workspace, workspace_bytes, (uint64_t)clip_workspace())) != NVFP4_OK)
    return st;
  DeviceInfo dev;
  if ((st = current_device(&dev)) != NVFP4_OK) return st;
  cudaError_t e = launch_clip(list.get(), count, clip, max_norm, norm, workspace, dev, stream);
  return e == cudaSuccess ? NVFP4_OK : cuda_fail(e, "clip launch");
}
}  // namespace

nvfp4_status nvfp4_grad_norm(const nvfp4_tensor* tensors, int32_t count, float* norm,
                             void* workspace, uint64_t workspace_bytes, nvfp4_stream_t stream) {
  return clip_impl(tensors, count, false, 0.0f, norm, workspace, workspace_bytes, stream);
}

nvfp4_status nvfp4_clip_grad_norm(const nvfp4_tensor* tensors, int32_t count, float max_norm,
                                  float* norm, void* workspace, uint64_t workspace_bytes,
                                  nvfp4_stream_t stream) {
  return clip_impl(tensors, count, true, max_norm, norm, workspace, workspace_bytes, stream);
}

}  // extern "C"
