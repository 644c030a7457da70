// rb_add_rms_norm: host checks and dispatch (rms_norm.cuh has the kernel).
#include "rms_norm.cuh"

namespace rb {
namespace norm {
// (in the translation units of their types)
extern template rb_status run_norm<__nv_bfloat16>(const NormArgs&, bool, cudaStream_t);
extern template rb_status run_norm<__half>(const NormArgs&, bool, cudaStream_t);
extern template rb_status run_norm<float>(const NormArgs&, bool, cudaStream_t);
}  // namespace norm
}  // namespace rb

extern "C" rb_status rb_add_rms_norm(int32_t num_rows, int32_t hidden_size, int32_t dtype,
                                     const void* d_x, int64_t x_stride, const void* d_residual,
                                     int64_t residual_stride, void* d_residual_out,
                                     int64_t residual_out_stride, const void* d_weight, float eps,
                                     int32_t out_dtype, int32_t group_size, void* d_out,
                                     float* d_scales, void* stream) {
  rb::CallRange range_("rb_add_rms_norm");
  using namespace rb;
  using namespace rb::norm;
  if (num_rows < 0 || hidden_size < 1 || !std::isfinite(eps) || eps < 0.f) return RB_ERR_INVALID_ARG;
  if (dtype != RB_BF16 && dtype != RB_FP16 && dtype != RB_FP32) return RB_ERR_UNSUPPORTED;
  const bool eight = out_dtype == RB_E4M3;
  if ((!eight && out_dtype != dtype) || hidden_size > kMostRuns * kRun) return RB_ERR_UNSUPPORTED;
  if (group_size != 0) {
    if (!eight || group_size < 0) return RB_ERR_INVALID_ARG;
    if (group_size != 16 && group_size != 32 && group_size != 64 && group_size != 128 &&
        group_size != 256)
      return RB_ERR_UNSUPPORTED;
    if (hidden_size % group_size != 0) return RB_ERR_INVALID_ARG;
  }
  const bool residual = d_residual != nullptr;
  if (residual != (d_residual_out != nullptr) || x_stride < hidden_size ||
      (residual && (residual_stride < hidden_size || residual_out_stride < hidden_size)))
    return RB_ERR_INVALID_ARG;
  if (num_rows == 0) return RB_OK;
  if (d_x == nullptr || d_weight == nullptr || d_out == nullptr || eight != (d_scales != nullptr))
    return RB_ERR_INVALID_ARG;
  const int size = dtype == RB_FP32 ? 4 : 2;
  auto element_aligned = [](const void* p, int bytes) {
    return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0;
  };
  if (!element_aligned(d_x, size) || !element_aligned(d_residual, size) ||
      !element_aligned(d_residual_out, size) || !element_aligned(d_weight, size) ||
      !element_aligned(d_out, eight ? 1 : size) || !element_aligned(d_scales, 4))
    return RB_ERR_INVALID_ARG;
  NormArgs a{};
  a.x = d_x;
  a.residual = d_residual;
  a.weight = d_weight;
  a.residual_out = d_residual_out;
  a.out = d_out;
  a.scales = d_scales;
  a.x_stride = x_stride;
  a.residual_stride = residual_stride;
  a.residual_out_stride = residual_out_stride;
  a.rows = num_rows;
  a.hidden = hidden_size;
  a.group = group_size;
  a.eps = eps;
  auto rows_aligned = [size](const void* p, int64_t stride) {
    return aligned16(p) && stride * size % 16 == 0;
  };
  a.wide = hidden_size % kRun == 0 && rows_aligned(d_x, x_stride) && aligned16(d_weight) &&
           (eight ? (reinterpret_cast<uintptr_t>(d_out) & 7u) == 0 : aligned16(d_out)) &&
           (!residual || (rows_aligned(d_residual, residual_stride) &&
                          rows_aligned(d_residual_out, residual_out_stride)));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == RB_BF16) return run_norm<__nv_bfloat16>(a, eight, s);
  if (dtype == RB_FP16) return run_norm<__half>(a, eight, s);
  return run_norm<float>(a, eight, s);
}
