// The residual's addition and the root-mean-square norm of rows of hidden states (rms_norm.cu has the
// entry point; one translation unit per type of row).  Not part of the C ABI.
//
//   r = x + residual (rounded to the rows' type),  y = r / sqrt(mean(r^2) + eps) * weight
//   8 bits: s = max |y| / 448 over the row or over each group, code = e4m3(y / s)
//
// Bound by HBM: a row is read once, held in registers between the sum of its squares and its
// output, and written once.  A thread holds two runs of eight values; a row is one warp's (up to 512
// values) or one CTA's.  The 8-bit codes need no norm: y / s = 448 z / max |z| with z = r weight, so
// one reduction gives the sum and the maximum.
//
// What it took (8192 x 4096 bf16 into 8 bits, 235 MB, passes back to back): values held as fp32 92
// us; as they lie in memory 64; z kept for the codes 52; rows of whole aligned runs without checks
// of each, the residual added two values at a time 38.  Issue was the limit, at a warp
// instruction a value, then a third of one.
#pragma once

#include <cuda_fp16.h>

#include "rb_internal.cuh"

namespace rb {
namespace norm {

constexpr int kRun = 8;          // values of one run
constexpr int kMostRuns = 4096;  // of a row
constexpr float kMax8 = 448.f;   // largest e4m3 value

enum Out : int { kPlain, kRowScales, kGroupScales };

struct NormArgs {
  const void *x, *residual, *weight;
  void *residual_out, *out;
  float* scales;
  long long x_stride, residual_stride, residual_out_stride;
  int rows, hidden, group;  // group 0: one scale a row
  float eps;
  int wide;  // every row is whole runs, aligned to 16 bytes (8 for 8-bit outputs)
};

template <class T>
rb_status run_norm(const NormArgs& a, bool eight, cudaStream_t s);

namespace {

// Eight values of a row as they lie in memory.
template <class T>
struct alignas(16) Run {
  T v[kRun];
};

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

// Both ways between a run and its fp32 values.
template <class T>
__device__ __forceinline__ void unpack(const Run<T>& r, float (&f)[kRun]) {
#pragma unroll
  for (int i = 0; i < kRun; ++i) f[i] = static_cast<float>(r.v[i]);
}
__device__ __forceinline__ void unpack(const Run<__nv_bfloat16>& r, float (&f)[kRun]) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(r.v);
#pragma unroll
  for (int i = 0; i < kRun / 2; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <class T>
__device__ __forceinline__ void pack(Run<T>& r, const float (&f)[kRun]) {
#pragma unroll
  for (int i = 0; i < kRun; ++i) r.v[i] = from_float<T>(f[i]);
}

// a + b.  Two 16-bit values at a time: rounded once, which for summands of 8 or 11 bits is what fp32
// gives when it is rounded again.
__device__ __forceinline__ void add(Run<float>& a, const Run<float>& b) {
#pragma unroll
  for (int i = 0; i < kRun; ++i) a.v[i] += b.v[i];
}
__device__ __forceinline__ void add(Run<__half>& a, const Run<__half>& b) {
  __half2* x = reinterpret_cast<__half2*>(a.v);
  const __half2* y = reinterpret_cast<const __half2*>(b.v);
#pragma unroll
  for (int i = 0; i < kRun / 2; ++i) x[i] = __hadd2(x[i], y[i]);
}
__device__ __forceinline__ void add(Run<__nv_bfloat16>& a, const Run<__nv_bfloat16>& b) {
  __nv_bfloat162* x = reinterpret_cast<__nv_bfloat162*>(a.v);
  const __nv_bfloat162* y = reinterpret_cast<const __nv_bfloat162*>(b.v);
#pragma unroll
  for (int i = 0; i < kRun / 2; ++i) x[i] = __hadd2(x[i], y[i]);
}

// Where a thread's i-th eight values are: a run, or, where rows are not whole aligned runs and no
// group of neighbours has to stay together, every threads-th value (so that a warp's are adjacent).
template <bool kSpread>
struct Span {
  int first, step, n;
  __device__ Span(int tid, int i, int threads, int n_)
      : first(kSpread ? i * kRun * threads + tid : (tid + i * threads) * kRun),
        step(kSpread ? threads : 1),
        n(n_) {}
  __device__ bool any() const { return first < n; }
  __device__ int at(int k) const { return first + k * step; }
};

// Its values (zeros past the end), and back.
template <class T, bool kWide, bool kSpread>
__device__ __forceinline__ Run<T> load_run(const T* row, const Span<kSpread>& p) {
  Run<T> r;
  if constexpr (kWide) {
    constexpr int kVec = static_cast<int>(sizeof(T)) * kRun / 16;
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      reinterpret_cast<uint4*>(r.v)[i] = reinterpret_cast<const uint4*>(row + p.first)[i];
  } else {
#pragma unroll
    for (int k = 0; k < kRun; ++k) r.v[k] = p.at(k) < p.n ? row[p.at(k)] : from_float<T>(0.f);
  }
  return r;
}
template <class T, bool kWide, bool kSpread>
__device__ __forceinline__ void store_run(T* row, const Span<kSpread>& p, const Run<T>& r) {
  if constexpr (kWide) {
    constexpr int kVec = static_cast<int>(sizeof(T)) * kRun / 16;
#pragma unroll
    for (int i = 0; i < kVec; ++i)
      reinterpret_cast<uint4*>(row + p.first)[i] = reinterpret_cast<const uint4*>(r.v)[i];
  } else {
#pragma unroll
    for (int k = 0; k < kRun; ++k)
      if (p.at(k) < p.n) row[p.at(k)] = r.v[k];
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

// A row is a CTA's: of kWarps warps, or (0) of as many as it has, kMost threads at most; with one warp a
// row, a CTA has four rows.
template <class T, int kWarps, int kMost, int kRuns, int kOut, bool kWide>
__global__ void __launch_bounds__(kMost,
                                  kMost == 1024 ? 1 : (sizeof(T) == 4 ? 1024 : 1536) / kMost)
    norm_kernel(const NormArgs a) {
  constexpr bool kRowScale = kOut == kRowScales;
  using Place = Span<!kWide && kOut != kGroupScales>;
  __shared__ float2 s_row[32];
  const int tid = kWarps == 1 ? threadIdx.x & 31 : threadIdx.x;
  const int row = kWarps == 1 ? blockIdx.x * 4 + (threadIdx.x >> 5) : blockIdx.x;
  if (row >= a.rows) return;  // (a whole warp, when a CTA has several rows)
  const int threads = kWarps > 0 ? kWarps * 32 : blockDim.x;
  const int n = a.hidden;
  const T* x = static_cast<const T*>(a.x) + row * a.x_stride;
  const T* weight = static_cast<const T*>(a.weight);
  auto place = [&](int i) { return Place(tid, i, threads, n); };
  Run<T> r[kRuns], w[kRuns];
#pragma unroll
  for (int i = 0; i < kRuns; ++i)
    if (place(i).any()) r[i] = load_run<T, kWide>(x, place(i));
  if (a.residual != nullptr) {
    const T* res = static_cast<const T*>(a.residual) + row * a.residual_stride;
    T* after = static_cast<T*>(a.residual_out) + row * a.residual_out_stride;
    Run<T> more[kRuns];
#pragma unroll
    for (int i = 0; i < kRuns; ++i)
      if (place(i).any()) more[i] = load_run<T, kWide>(res, place(i));
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
      if (!place(i).any()) break;
      add(r[i], more[i]);
      store_run<T, kWide>(after, place(i), r[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < kRuns; ++i)
    if (place(i).any()) w[i] = load_run<T, kWide>(weight, place(i));
  float sum = 0.f, top = 0.f;
  float z[kRuns][kRun];  // r, in 8 bits r weight
#pragma unroll
  for (int i = 0; i < kRuns; ++i) {
    if (!place(i).any()) {
#pragma unroll
      for (int k = 0; k < kRun; ++k) z[i][k] = 0.f;
      continue;
    }
    unpack(r[i], z[i]);
#pragma unroll
    for (int k = 0; k < kRun; ++k) sum = fmaf(z[i][k], z[i][k], sum);
    if constexpr (kOut != kPlain) {
      float f[kRun];
      unpack(w[i], f);
#pragma unroll
      for (int k = 0; k < kRun; ++k) {
        z[i][k] *= f[k];
        if constexpr (kRowScale) top = fmaxf(top, fabsf(z[i][k]));
      }
    }
  }
  const float2 both = row_reduce<kWarps, kRowScale>(sum, top, s_row);
  const float inv = rsqrtf(both.x / static_cast<float>(n) + a.eps);
  if constexpr (kOut == kPlain) {
    T* out = static_cast<T*>(a.out) + static_cast<size_t>(row) * n;
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
      if (!place(i).any()) break;
      float f[kRun];
      unpack(w[i], f);
#pragma unroll
      for (int k = 0; k < kRun; ++k) z[i][k] = z[i][k] * inv * f[k];
      pack(r[i], z[i]);
      store_run<T, kWide>(out, place(i), r[i]);
    }
  } else {
    uint8_t* out = static_cast<uint8_t*>(a.out) + static_cast<size_t>(row) * n;
    const int lanes = a.group / kRun;  // of one group
    top = both.y;
#pragma unroll
    for (int i = 0; i < kRuns; ++i) {
      const Place p = place(i);
      if constexpr (!kRowScale) {  // (every lane of the warp is here: a group ends with the row)
        top = 0.f;
#pragma unroll
        for (int k = 0; k < kRun; ++k) top = fmaxf(top, fabsf(z[i][k]));
        for (int o = lanes / 2; o > 0; o >>= 1)
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
      }
      if (!p.any()) continue;
      const float s = top * inv * (1.f / kMax8);
      float most = top;
      if (most < 0x1p-100f) {  // (448 / most would pass fp32's range)
        most *= 0x1p100f;
#pragma unroll
        for (int k = 0; k < kRun; ++k) z[i][k] *= 0x1p100f;
      }
      // codes are 0 where s is, and NaN where s or the value is
      const float by = s > 0.f && most < INFINITY ? kMax8 / most : s * 0.f;
#pragma unroll
      for (int k = 0; k < kRun; ++k) z[i][k] *= by;
      const uint2 c = codes8(z[i]);
      if constexpr (kWide) {
        *reinterpret_cast<uint2*>(out + p.first) = c;
      } else {
        const uint8_t* b = reinterpret_cast<const uint8_t*>(&c);
#pragma unroll
        for (int k = 0; k < kRun; ++k)
          if (p.at(k) < n) out[p.at(k)] = b[k];
      }
      if constexpr (kRowScale) {
        if (p.first == 0) a.scales[row] = s;
      } else if (p.first % a.group == 0) {
        a.scales[static_cast<size_t>(row) * (n / a.group) + p.first / a.group] = s;
      }
    }
  }
}

// Two runs a thread, in whole warps, up to a CTA of 1024 (four beyond).  For rows of whole aligned
// runs a count of warps that is a power of two is compiled in (8192 x 4096 bf16 into 8 bits, cold: 36 us
// against 38).  Four runs on half the threads are equal there, and 2047 x 5120 fp16 in groups takes
// 21.6 instead of 19.6; persistent CTAs that load the next row ahead took 65 where this took 44.
// Rows that are not whole aligned runs go one value at a time: 8192 x 4096 bf16, rows 4157 apart,
// 71 us instead of 40, into 8 bits 75 instead of 36.
//
// Four runs are held in the 64 registers that a CTA of 1024 leaves: above 16384 values fp32 rows spill
// 112 to 292 bytes a thread (1024 x 32768 fp32 124 us, 0.64 of the copy rate; bf16, 16 at most, 0.75).
// Unaligned fp16 and bf16 rows of up to 8192 values spill 4 to 52 bytes in the 40 registers of their
// three CTAs an SM.
template <class T, int kOut>
rb_status launch_norm(const NormArgs& a, cudaStream_t s) {
  const int runs = (a.hidden + kRun - 1) / kRun;
  const int warps = (runs + 63) / 64, rows = a.rows;
  if (a.wide) {
    if (warps == 1) norm_kernel<T, 1, 128, 2, kOut, true><<<(rows - 1) / 4 + 1, 128, 0, s>>>(a);
    else if (warps == 2) norm_kernel<T, 2, 64, 2, kOut, true><<<rows, 64, 0, s>>>(a);
    else if (warps == 4) norm_kernel<T, 4, 128, 2, kOut, true><<<rows, 128, 0, s>>>(a);
    else if (warps == 8) norm_kernel<T, 8, 256, 2, kOut, true><<<rows, 256, 0, s>>>(a);
    else if (warps == 16) norm_kernel<T, 16, 512, 2, kOut, true><<<rows, 512, 0, s>>>(a);
    else if (warps < 16) norm_kernel<T, 0, 512, 2, kOut, true><<<rows, warps * 32, 0, s>>>(a);
    else if (warps <= 32) norm_kernel<T, 0, 1024, 2, kOut, true><<<rows, warps * 32, 0, s>>>(a);
    else norm_kernel<T, 0, 1024, 4, kOut, true><<<rows, (warps + 1) / 2 * 32, 0, s>>>(a);
  } else {
    if (warps == 1) norm_kernel<T, 1, 128, 2, kOut, false><<<(rows - 1) / 4 + 1, 128, 0, s>>>(a);
    else if (warps <= 16) norm_kernel<T, 0, 512, 2, kOut, false><<<rows, warps * 32, 0, s>>>(a);
    else if (warps <= 32) norm_kernel<T, 0, 1024, 2, kOut, false><<<rows, warps * 32, 0, s>>>(a);
    else norm_kernel<T, 0, 1024, 4, kOut, false><<<rows, (warps + 1) / 2 * 32, 0, s>>>(a);
  }
  if (last_launch_status() != RB_OK) return RB_ERR_CUDA;
  note_launches(1);
  return RB_OK;
}

}  // namespace

template <class T>
rb_status run_norm(const NormArgs& a, bool eight, cudaStream_t s) {
  if (!eight) return launch_norm<T, kPlain>(a, s);
  return a.group == 0 ? launch_norm<T, kRowScales>(a, s) : launch_norm<T, kGroupScales>(a, s);
}

}  // namespace norm
}  // namespace rb
