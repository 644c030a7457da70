// rb_add_rms_norm: the residual's addition and the root-mean-square norm of rows of hidden states,
// with an output in the rows' type or in 8 bits with scales.
//
//   r = x + residual (rounded to the rows' type),  y = r / sqrt(mean(r^2) + eps) * weight
//   8 bits: s = max |y| / 448 over the row or over each group, code = e4m3(y / s)
//
// Bound by HBM: a row is read once, held in registers between the sum of its squares and its
// output, and written once.  A thread holds runs of eight values; a row is one warp's (up to 1024
// values) or one CTA's.
#include <cuda_fp16.h>

#include "rb_internal.cuh"

namespace rb {
namespace {

constexpr int kRun = 8;        // values of one run
constexpr int kRuns = 4;       // runs a thread may hold
constexpr float kMax8 = 448.f; // largest e4m3 value

struct NormArgs {
  const void *x, *residual, *weight;
  void *residual_out, *out;
  float* scales;
  long long x_stride, residual_stride, residual_out_stride;
  int rows, hidden, group;  // group 0: one scale a row
  float eps;
  int wide;  // x, residual and residual_out take 16-byte accesses
};

template <class T>
__device__ __forceinline__ float to_float(T v) {
  return static_cast<float>(v);
}
template <class T>
__device__ __forceinline__ T from_float(float f);
template <>
__device__ __forceinline__ float from_float<float>(float f) {
  return f;
}
template <>
__device__ __forceinline__ __half from_float<__half>(float f) {
  return __float2half_rn(f);
}
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float f) {
  return __float2bfloat16_rn(f);
}

// Run `run` of a row of n values: eight values, zeros past the end.
template <class T>
__device__ __forceinline__ void load_run(const T* row, int run, int n, bool wide, float (&f)[kRun]) {
  const T* p = row + run * kRun;
  if (wide && (run + 1) * kRun <= n) {
    constexpr int kVec = static_cast<int>(sizeof(T)) * kRun / 16;
    uint4 w[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) w[i] = reinterpret_cast<const uint4*>(p)[i];
    const T* v = reinterpret_cast<const T*>(w);
#pragma unroll
    for (int i = 0; i < kRun; ++i) f[i] = to_float(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < kRun; ++i) f[i] = run * kRun + i < n ? to_float(p[i]) : 0.f;
  }
}

template <class T>
__device__ __forceinline__ void store_run(T* row, int run, int n, bool wide, const float (&f)[kRun]) {
  T* p = row + run * kRun;
  if (wide && (run + 1) * kRun <= n) {
    constexpr int kVec = static_cast<int>(sizeof(T)) * kRun / 16;
    uint4 w[kVec];
    T* v = reinterpret_cast<T*>(w);
#pragma unroll
    for (int i = 0; i < kRun; ++i) v[i] = from_float<T>(f[i]);
#pragma unroll
    for (int i = 0; i < kVec; ++i) reinterpret_cast<uint4*>(p)[i] = w[i];
  } else {
#pragma unroll
    for (int i = 0; i < kRun; ++i)
      if (run * kRun + i < n) p[i] = from_float<T>(f[i]);
  }
}

// Eight e4m3 codes (nearest, ties to even, 448 at most), value 0 in the lowest byte.
__device__ __forceinline__ uint2 codes8(const float (&f)[kRun]) {
  uint16_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h[i]) : "f"(f[2 * i + 1]), "f"(f[2 * i]));
  return make_uint2(h[0] | static_cast<uint32_t>(h[1]) << 16,
                    h[2] | static_cast<uint32_t>(h[3]) << 16);
}

// Reduction over the `kWarps` warps of a row; every thread gets the result.
template <int kWarps, class Op>
__device__ __forceinline__ float row_reduce(float v, float* shared, const Op& op) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  if constexpr (kWarps > 1) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) shared[threadIdx.x >> 5] = v;
    __syncthreads();
    v = shared[lane % kWarps];
#pragma unroll
    for (int o = kWarps / 2; o > 0; o >>= 1) v = op(v, __shfl_xor_sync(0xffffffffu, v, o));
  }
  return v;
}

template <class T, int kWarps, bool k8bit>
__global__ void __launch_bounds__(kWarps == 1 ? 128 : kWarps * 32) norm_kernel(const NormArgs a) {
  __shared__ float s_sum[32], s_max[32];
  const int tid = kWarps == 1 ? static_cast<int>(threadIdx.x & 31) : static_cast<int>(threadIdx.x);
  const int row = kWarps == 1 ? blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
  if (row >= a.rows) return;  // (a whole warp, when a CTA has several rows)
  constexpr int kThreads = kWarps * 32;
  const int n = a.hidden;
  const bool wide = a.wide != 0;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  float y[kRuns][kRun];
#pragma unroll
  for (int i = 0; i < kRuns; ++i) {
    const int run = tid + i * kThreads;
    if (run * kRun < n) load_run(x, run, n, wide, y[i]);
    else
#pragma unroll
      for (int k = 0; k < kRun; ++k) y[i][k] = 0.f;
  }
  if (a.residual != nullptr) {
    const T* res = static_cast<const T*>(a.residual) + row * a.residual_stride;
    T* after = static_cast<T*>(a.residual_out) + row * a.residual_out_stride;
    float z[kRuns][kRun];
#pragma unroll
    for (int i = 0; i < kRuns; ++i)
      if ((tid + i * kThreads) * kRun < n) load_run(res, tid + i * kThreads, n, wide, z[i]);
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
      const int run = tid + i * kThreads;
      if (run * kRun >= n) break;
#pragma unroll
      for (int k = 0; k < kRun; ++k) y[i][k] = to_float(from_float<T>(y[i][k] + z[i][k]));
      store_run(after, run, n, wide, y[i]);
    }
  }
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < kRuns; ++i)
#pragma unroll
    for (int k = 0; k < kRun; ++k) sum = fmaf(y[i][k], y[i][k], sum);
  sum = row_reduce<kWarps>(sum, s_sum, [](float p, float q) { return p + q; });
  const float inv = rsqrtf(sum / static_cast<float>(n) + a.eps);
  const T* weight = static_cast<const T*>(a.weight);
  const bool weight_wide = aligned16(a.weight);
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < kRuns; ++i) {
    const int run = tid + i * kThreads;
    if (run * kRun >= n) break;
    float w[kRun];
    load_run(weight, run, n, weight_wide, w);
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      y[i][k] = y[i][k] * inv * w[k];
      if constexpr (k8bit) top = fmaxf(top, fabsf(y[i][k]));
    }
    if constexpr (!k8bit) {
      T* out = static_cast<T*>(a.out) + static_cast<size_t>(row) * n;
      store_run(out, run, n, aligned16(out), y[i]);
    }
  }
  if constexpr (k8bit) {
    uint8_t* out = static_cast<uint8_t*>(a.out) + static_cast<size_t>(row) * n;
    const bool out_wide = (reinterpret_cast<uintptr_t>(out) & 7u) == 0;
    if (a.group == 0)
      top = row_reduce<kWarps>(top, s_max, [](float p, float q) { return fmaxf(p, q); });
    const int lanes = a.group / kRun;  // of one group
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
      const int run = tid + i * kThreads;
      if (a.group != 0) {  // (every lane of the warp is here: a group ends with the row)
        top = 0.f;
#pragma unroll
        for (int k = 0; k < kRun; ++k) top = fmaxf(top, fabsf(y[i][k]));
        for (int o = lanes / 2; o > 0; o >>= 1)
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      }
      if (run * kRun >= n) continue;
      const float s = top / kMax8;
      float t[kRun];
#pragma unroll
      for (int k = 0; k < kRun; ++k)  // (0 where s is 0, but NaN stays NaN)
        t[k] = s > 0.f ? __fdiv_rn(y[i][k], s) : y[i][k] * 0.f;
      const uint2 c = codes8(t);
      if (out_wide && (run + 1) * kRun <= n) {
        *reinterpret_cast<uint2*>(out + run * kRun) = c;
      } else {
        const uint8_t* b = reinterpret_cast<const uint8_t*>(&c);
        for (int k = 0; k < kRun; ++k)
          if (run * kRun + k < n) out[run * kRun + k] = b[k];
      }
      if (a.group == 0) {
        if (run == 0) a.scales[row] = s;
      } else if (run % lanes == 0) {
        a.scales[static_cast<size_t>(row) * (n / a.group) + run / lanes] = s;
      }
    }
  }
}

template <class T, bool k8bit>
void launch_norm(const NormArgs& a, cudaStream_t s) {
  const int runs = (a.hidden + kRun - 1) / kRun;
  if (runs <= 32 * kRuns) norm_kernel<T, 1, k8bit><<<(a.rows + 3) / 4, 128, 0, s>>>(a);
  else if (runs <= 128 * kRuns) norm_kernel<T, 4, k8bit><<<a.rows, 128, 0, s>>>(a);
  else if (runs <= 256 * kRuns) norm_kernel<T, 8, k8bit><<<a.rows, 256, 0, s>>>(a);
  else if (runs <= 512 * kRuns) norm_kernel<T, 16, k8bit><<<a.rows, 512, 0, s>>>(a);
  else norm_kernel<T, 32, k8bit><<<a.rows, 1024, 0, s>>>(a);
}

template <class T>
rb_status run_norm(const NormArgs& a, bool eight, cudaStream_t s) {
  if (eight) launch_norm<T, true>(a, s);
  else launch_norm<T, false>(a, s);
  if (last_launch_status() != RB_OK) return RB_ERR_CUDA;
  note_launches(1);
  return RB_OK;
}

}  // namespace
}  // namespace rb

extern "C" rb_status rb_add_rms_norm(int32_t num_rows, int32_t hidden_size, int32_t dtype,
                                     const void* d_x, int64_t x_stride, const void* d_residual,
                                     int64_t residual_stride, void* d_residual_out,
                                     int64_t residual_out_stride, const void* d_weight, float eps,
                                     int32_t out_dtype, int32_t group_size, void* d_out,
                                     float* d_scales, void* stream) {
  rb::CallRange range_("rb_add_rms_norm");
  using namespace rb;
  if (num_rows < 0 || hidden_size < 1 || !std::isfinite(eps) || eps < 0.f) return RB_ERR_INVALID_ARG;
  if (dtype != RB_BF16 && dtype != RB_FP16 && dtype != RB_FP32) return RB_ERR_UNSUPPORTED;
  const bool eight = out_dtype == RB_E4M3;
  if ((!eight && out_dtype != dtype) || hidden_size > 1024 * kRuns * kRun) return RB_ERR_UNSUPPORTED;
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
  a.wide = rows_aligned(d_x, x_stride) &&
           (!residual || (rows_aligned(d_residual, residual_stride) &&
                          rows_aligned(d_residual_out, residual_out_stride)));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == RB_BF16) return run_norm<__nv_bfloat16>(a, eight, s);
  if (dtype == RB_FP16) return run_norm<__half>(a, eight, s);
  return run_norm<float>(a, eight, s);
}
