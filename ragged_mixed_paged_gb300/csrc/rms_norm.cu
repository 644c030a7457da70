// rb_add_rms_norm: the residual's addition and the root-mean-square norm of rows of hidden states,
// with an output in the rows' type or in 8 bits with scales.
//
//   r = x + residual (rounded to the rows' type),  y = r / sqrt(mean(r^2) + eps) * weight
//   8 bits: s = max |y| / 448 over the row or over each group, code = e4m3(y / s)
//
// Bound by HBM: a row is read once, held in registers between the sum of its squares and its
// output, and written once.  A thread holds runs of eight values; a row is one warp's (up to 1024
// values) or one CTA's.
#include "kv4.cuh"

namespace rb {
namespace {

constexpr int kRun = 8;        // values of one run
constexpr int kMostRuns = 4096;  // of a row
constexpr float kMax8 = 448.f; // largest e4m3 value

enum Out : int { kPlain, kRowScales, kGroupScales };

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

// Eight values of a row as they lie in memory.
template <class T>
struct alignas(16) Run {
  T v[kRun];
};

// Run `run` of a row of n values, zeros past the end.
template <class T>
__device__ __forceinline__ Run<T> load_run(const T* row, int run, int n, bool wide) {
  const T* p = row + run * kRun;
  Run<T> r;
  if (wide && (run + 1) * kRun <= n) {
    constexpr int kVec = static_cast<int>(sizeof(T)) * kRun / 16;
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      reinterpret_cast<uint4*>(r.v)[i] = reinterpret_cast<const uint4*>(p)[i];
  } else {
#pragma unroll
    for (int i = 0; i < kRun; ++i) r.v[i] = run * kRun + i < n ? p[i] : from_float<T>(0.f);
  }
  return r;
}

template <class T>
__device__ __forceinline__ void store_run(T* row, int run, int n, bool wide, const Run<T>& r) {
  T* p = row + run * kRun;
  if (wide && (run + 1) * kRun <= n) {
    constexpr int kVec = static_cast<int>(sizeof(T)) * kRun / 16;
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(r.v)[i];
  } else {
#pragma unroll
    for (int i = 0; i < kRun; ++i)
      if (run * kRun + i < n) p[i] = r.v[i];
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

// Sum and maximum over the warps of a row (kWarps of them; 0: the CTA's); every thread gets both.
template <int kWarps, bool kMax>
__device__ __forceinline__ float2 row_reduce(float sum, float top, float2* shared) {
  auto over_lanes = [&](int first) {
#pragma unroll
    for (int o = first; o > 0; o >>= 1) {
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if (kMax) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    }
  };
  over_lanes(16);
  if constexpr (kWarps != 1) {
    const int lane = threadIdx.x & 31;
    if (lane == 0) shared[threadIdx.x >> 5] = make_float2(sum, top);
    __syncthreads();
    float2 v = make_float2(0.f, 0.f);
    if (kWarps > 0) v = shared[lane % (kWarps > 0 ? kWarps : 1)];
    else if (lane < blockDim.x / 32) v = shared[lane];
    sum = v.x;
    top = v.y;
    over_lanes(kWarps > 0 ? kWarps / 2 : 16);
  }
  return make_float2(sum, top);
}

// The 8-bit codes need no norm: y / (max |y| / 448) is 448 z / max |z| with z = r weight, which is
// exact in fp32 for 16-bit types.  So ties are ties, and one reduction gives sum and maximum.
// A row is a CTA's: of kWarps warps, or (0) of as many as it has, kMost threads at most; with one warp a
// row, a CTA has four rows.
template <class T, int kWarps, int kMost, int kRuns, int kOut>
__global__ void __launch_bounds__(kMost, kMost == 1024 ? 1 : 1536 / kMost)
    norm_kernel(const NormArgs a) {
  constexpr bool k8bit = kOut != kPlain, kRowScale = kOut == kRowScales;
  __shared__ float2 s_row[32];
  const int tid = kWarps == 1 ? threadIdx.x & 31 : threadIdx.x;
  const int row = kWarps == 1 ? blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
  if (row >= a.rows) return;  // (a whole warp, when a CTA has several rows)
  const int threads = kWarps > 0 ? kWarps * 32 : blockDim.x;
  const int n = a.hidden;
  const bool wide = a.wide != 0;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const T* weight = static_cast<const T*>(a.weight);
  const bool weight_wide = aligned16(a.weight);
  Run<T> y[kRuns];
#pragma unroll
  for (int i = 0; i < kRuns; ++i)
    if ((tid + i * threads) * kRun < n) y[i] = load_run(x, tid + i * threads, n, wide);
  if (a.residual != nullptr) {
    const T* res = static_cast<const T*>(a.residual) + row * a.residual_stride;
    T* after = static_cast<T*>(a.residual_out) + row * a.residual_out_stride;
    Run<T> r[kRuns];
#pragma unroll
    for (int i = 0; i < kRuns; ++i)
      if ((tid + i * threads) * kRun < n) r[i] = load_run(res, tid + i * threads, n, wide);
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
      const int run = tid + i * threads;
      if (run * kRun >= n) break;
#pragma unroll
      for (int k = 0; k < kRun; ++k)
        y[i].v[k] = from_float<T>(to_float(y[i].v[k]) + to_float(r[i].v[k]));
      store_run(after, run, n, wide, y[i]);
    }
  }
  float sum = 0.f, top = 0.f;
  float z[kRuns][kRun];
#pragma unroll
  for (int i = 0; i < kRuns; ++i) {
    const int run = tid + i * threads;
    if (run * kRun >= n) break;
#pragma unroll
    for (int k = 0; k < kRun; ++k) {
      const float v = to_float(y[i].v[k]);
      sum = fmaf(v, v, sum);
    }
    if constexpr (kRowScale) {
      const Run<T> w = load_run(weight, run, n, weight_wide);
#pragma unroll
      for (int k = 0; k < kRun; ++k) {
        z[i][k] = to_float(y[i].v[k]) * to_float(w.v[k]);
        top = fmaxf(top, fabsf(z[i][k]));
      }
    }
  }
  const float2 both = row_reduce<kWarps, kRowScale>(sum, top, s_row);
  const float inv = rsqrtf(both.x / static_cast<float>(n) + a.eps);
  if constexpr (!k8bit) {
    T* out = static_cast<T*>(a.out) + static_cast<size_t>(row) * n;
    const bool out_wide = aligned16(out);
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
      const int run = tid + i * threads;
      if (run * kRun >= n) break;
      const Run<T> w = load_run(weight, run, n, weight_wide);
#pragma unroll
      for (int k = 0; k < kRun; ++k)
        y[i].v[k] = from_float<T>(to_float(y[i].v[k]) * inv * to_float(w.v[k]));
      store_run(out, run, n, out_wide, y[i]);
    }
  } else {
    uint8_t* out = static_cast<uint8_t*>(a.out) + static_cast<size_t>(row) * n;
    const bool out_wide = (reinterpret_cast<uintptr_t>(out) & 7u) == 0;
    const int lanes = a.group / kRun;  // of one group
    top = both.y;
    float r = __frcp_rn(top);
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
      const int run = tid + i * threads;
      const bool here = run * kRun < n;
      if constexpr (!kRowScale) {
        top = 0.f;
        if (here) {
          const Run<T> w = load_run(weight, run, n, weight_wide);
#pragma unroll
          for (int k = 0; k < kRun; ++k) {
            z[i][k] = to_float(y[i].v[k]) * to_float(w.v[k]);
            top = fmaxf(top, fabsf(z[i][k]));
          }
        }
        // (every lane of the warp is here: a group ends with the row)
        for (int o = lanes / 2; o > 0; o >>= 1)
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        r = __frcp_rn(top);
      }
      if (!here) continue;
      const float s = top * inv * (1.f / kMax8);
      const bool ordinary = s > 0.f && top < INFINITY && r < INFINITY;
#pragma unroll
      for (int k = 0; k < kRun; ++k)  // (0 where s is 0, but NaN stays NaN)
        z[i][k] = ordinary ? kv4::quotient(z[i][k] * kMax8, top, r) : z[i][k] * inv * 0.f;
      const uint2 c = codes8(z[i]);
      if (out_wide && (run + 1) * kRun <= n) {
        *reinterpret_cast<uint2*>(out + run * kRun) = c;
      } else {
        const uint8_t* b = reinterpret_cast<const uint8_t*>(&c);
        for (int k = 0; k < kRun; ++k)
          if (run * kRun + k < n) out[run * kRun + k] = b[k];
      }
      if constexpr (kRowScale) {
        if (run == 0) a.scales[row] = s;
      } else if (run % lanes == 0) {
        a.scales[static_cast<size_t>(row) * (n / a.group) + run / lanes] = s;
      }
    }
  }
}

template <class T, int kOut>
rb_status run_norm(const NormArgs& a, cudaStream_t s) {
  // Two runs a thread, in whole warps, up to a CTA of 1024 (four beyond).  A count of warps that is
  // a power of two is compiled in (8192 x 4096 bf16 into 8 bits: 44 us against 49).  Four runs on
  // half the threads take 54 there; persistent CTAs that load the next row ahead 65.
  const int runs = (a.hidden + kRun - 1) / kRun;
  const int warps = (runs + 63) / 64;
  if (warps == 1) norm_kernel<T, 1, 128, 2, kOut><<<(a.rows + 3) / 4, 128, 0, s>>>(a);
  else if (warps == 2) norm_kernel<T, 2, 64, 2, kOut><<<a.rows, 64, 0, s>>>(a);
  else if (warps == 4) norm_kernel<T, 4, 128, 2, kOut><<<a.rows, 128, 0, s>>>(a);
  else if (warps == 8) norm_kernel<T, 8, 256, 2, kOut><<<a.rows, 256, 0, s>>>(a);
  else if (warps == 16) norm_kernel<T, 16, 512, 2, kOut><<<a.rows, 512, 0, s>>>(a);
  else if (warps < 16) norm_kernel<T, 0, 512, 2, kOut><<<a.rows, warps * 32, 0, s>>>(a);
  else if (warps <= 32) norm_kernel<T, 0, 1024, 2, kOut><<<a.rows, warps * 32, 0, s>>>(a);
  else norm_kernel<T, 0, 1024, 4, kOut><<<a.rows, (warps + 1) / 2 * 32, 0, s>>>(a);
  if (last_launch_status() != RB_OK) return RB_ERR_CUDA;
  note_launches(1);
  return RB_OK;
}

template <class T>
rb_status run_norm(const NormArgs& a, bool eight, cudaStream_t s) {
  if (!eight) return run_norm<T, kPlain>(a, s);
  return a.group == 0 ? run_norm<T, kRowScales>(a, s) : run_norm<T, kGroupScales>(a, s);
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
  a.wide = rows_aligned(d_x, x_stride) &&
           (!residual || (rows_aligned(d_residual, residual_stride) &&
                          rows_aligned(d_residual_out, residual_out_stride)));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (dtype == RB_BF16) return run_norm<__nv_bfloat16>(a, eight, s);
  if (dtype == RB_FP16) return run_norm<__half>(a, eight, s);
  return run_norm<float>(a, eight, s);
}
