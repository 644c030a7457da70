// rb_token_logprobs: log probability and rank of one given token per row of logits, the entropy
// of the row's distribution, and its most likely tokens.
//
// For a row x of V logits with m = max x and Z = sum exp(x_i - m):
//     log p_i = (x_i - m) - ln Z                    rank(t) = 1 + #{i : x_i > x_t}
//     H       = ln Z - (1/Z) sum exp(x_i - m) (x_i - m)
// and the top k of x, ordered by value, equal values by index.
//
// One pass over the row: with a running reference r, t_i = (x_i - r) log2(e) and e_i = 2^t_i,
// every thread keeps s = sum e_i and w = sum e_i t_i (both in fp32; a move of the reference by
// d log2 units maps them to s 2^-d and (w - d s) 2^-d), the count of x_i > x_t and the largest
// x_i it saw.  ln Z and H follow from s and w.  The difference comes before the factor, so the
// terms that matter (x_i near r) keep their bits however large the logits are.
//
// The top k takes no part in that loop but the threads' maxima: the k-th largest maximum of
// 128 lane groups bounds the k-th largest logit from below, only threads whose maximum reaches
// it hold candidates, and their share of the row (about k of 512) is read again, from L2.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include "rb_internal.cuh"

namespace rb {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kGroups = 128;      // lane groups (of 4 threads) whose maxima bound the k-th logit
constexpr int kMaxTop = 32;
constexpr int kMaxSplits = 8;     // CTAs of a cluster that share one row
constexpr int kCandidates = 1024;
constexpr int kBatch = 4;         // 16-byte loads in flight per thread
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// Differences to the reference are taken as at least kFar, so that masked (-inf) logits add
// 2^t t = 0 rather than 0 * inf.
constexpr float kFar = -1e30f;
constexpr float kLowest = -3.402823466e38f;  // the reference while a thread saw nothing finite
// The reference moves when a logit exceeds it by kGrowth: s <= V e^11 stays far inside fp32.
constexpr float kGrowth = 11.f;

struct LogprobArgs {
  const void* logits;
  long long row_stride;
  const int32_t* tokens;
  int rows, vocab, top;
  float* logprobs;
  int32_t* ranks;
  float* entropy;
  int32_t* top_ids;
  float* top_logprobs;
  int32_t* err;
};

__device__ __forceinline__ float max_nan(float a, float b) {  // NaN if either is
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

template <class T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kPer = 4;
  static __device__ __forceinline__ float one(const float* p) { return __ldg(p); }
  static __device__ __forceinline__ void unpack(const uint4& u, float2 (&x)[2]) {
    x[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
    x[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
  }
};
template <>
struct Elem<__nv_bfloat16> {
  static constexpr int kPer = 8;
  static __device__ __forceinline__ float one(const __nv_bfloat16* p) {
    return __uint_as_float(
        static_cast<uint32_t>(__ldg(reinterpret_cast<const unsigned short*>(p))) << 16);
  }
  static __device__ __forceinline__ float2 two(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ void unpack(const uint4& u, float2 (&x)[4]) {
    x[0] = two(u.x);
    x[1] = two(u.y);
    x[2] = two(u.z);
    x[3] = two(u.w);
  }
};
template <>
struct Elem<__half> {
  static constexpr int kPer = 8;
  static __device__ __forceinline__ float one(const __half* p) {
    return __half2float(__ushort_as_half(__ldg(reinterpret_cast<const unsigned short*>(p))));
  }
  static __device__ __forceinline__ float2 two(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  static __device__ __forceinline__ void unpack(const uint4& u, float2 (&x)[4]) {
    x[0] = two(u.x);
    x[1] = two(u.y);
    x[2] = two(u.z);
    x[3] = two(u.w);
  }
};

// s = sum 2^t, w = sum 2^t t with t = (x - ref) log2(e).
struct Sums {
  float ref, s, w;
  __device__ __forceinline__ void move_to(float to) {  // to >= ref
    if (s == 0.f) {
      w = 0.f;
    } else {
      const float d = fminf((to - ref) * kLog2e, -kFar), f = fast_exp2(-d);
      w = (w - d * s) * f;
      s *= f;
    }
    ref = to;
  }
  __device__ __forceinline__ void merge(Sums o) {
    const float to = fmaxf(ref, o.ref);
    move_to(to);
    o.move_to(to);
    s += o.s;
    w += o.w;
  }
};

struct Entry {
  float x;
  int i;
};
__device__ __forceinline__ bool before(const Entry& a, const Entry& b) {  // a ranks before b
  return a.x > b.x || (a.x == b.x && a.i < b.i);
}

struct Part {  // what one CTA of a row's cluster found
  Sums sums;
  float max;
  int above, top;
};

struct Shared {
  Part warp[kWarps];
  Part part;
  Entry best[kMaxTop];
  alignas(16) float group_max[kGroups];  // read four at a time
  float tau;
  int n_threads, n_cand, found, fill;
  unsigned short threads[kThreads];
  Entry cand[kCandidates];
  Entry red[kWarps];
  int warp_count[kWarps];
  Entry merged[kMaxSplits * kMaxTop];
};

// One CTA's part of a row: 16-byte vectors [v0, v1) of the row's aligned vectors.
template <class T>
struct Slice {
  using E = Elem<T>;
  const T* row;
  int vocab, off, v0, v1;  // off: elements of vector 0 that lie before the row

  __device__ __forceinline__ int first(int v) const { return v * E::kPer - off; }
  __device__ __forceinline__ bool whole(int v) const {
    return first(v) >= 0 && first(v) + E::kPer <= vocab;
  }
  __device__ __forceinline__ uint4 load(int v) const {
    return __ldg(reinterpret_cast<const uint4*>(row + first(v)));
  }
  __device__ __forceinline__ int lo() const { return max(0, first(v0)); }
  __device__ __forceinline__ int hi() const { return min(vocab, first(v1)); }
  // fn(x, index) for each element of vector v that is in the row
  template <class F>
  __device__ __forceinline__ void each(int v, F&& fn) const {
    if (whole(v)) {
      float2 x[E::kPer / 2];
      E::unpack(load(v), x);
#pragma unroll
      for (int k = 0; k < E::kPer / 2; ++k) {
        fn(x[k].x, first(v) + 2 * k);
        fn(x[k].y, first(v) + 2 * k + 1);
      }
    } else {
      for (int i = max(0, first(v)); i < min(vocab, first(v) + E::kPer); ++i)
        fn(E::one(row + i), i);
    }
  }
};

// The top entries of a slice in order, into sh.best; returns how many (min(k, elements)).
// `mine`: the largest element this thread read (vectors v0 + tid, + kThreads, ...).
template <class T>
__device__ int slice_top(const Slice<T>& sl, int k, float mine, Shared& sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int count = max(0, sl.hi() - sl.lo());
  const int want = min(k, count);
  if (want == 0) return 0;
  float g = mine;
  g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 1));
  g = fmaxf(g, __shfl_xor_sync(0xffffffffu, g, 2));
  if ((lane & 3) == 0) sh.group_max[tid >> 2] = g;
  if (tid == 0) sh.n_threads = sh.n_cand = 0;
  __syncthreads();
  if (tid < kGroups) {
    const float x = sh.group_max[tid];
    int rank = 0;
#pragma unroll 4
    for (int j = 0; j < kGroups; j += 4) {
      const float4 o = *reinterpret_cast<const float4*>(sh.group_max + j);
      rank += (o.x > x) + (o.y > x) + (o.z > x) + (o.w > x);
      rank += (o.x == x && j < tid) + (o.y == x && j + 1 < tid) + (o.z == x && j + 2 < tid) +
              (o.w == x && j + 3 < tid);
    }
    if (rank == want - 1) sh.tau = x;
  }
  __syncthreads();
  const float tau = sh.tau;  // at least `want` elements are >= tau (-inf: fewer groups had any)
  // Many elements equal to tau (masked logits above all): take those above it, then the first
  // equal ones in the order of their index.
  const bool many = tau == -INFINITY;
  if (mine > tau || (!many && mine == tau))
    sh.threads[atomicAdd(&sh.n_threads, 1)] = static_cast<unsigned short>(tid);
  __syncthreads();
  const int n_threads = sh.n_threads;
  const int per = (sl.v1 - sl.v0 + kThreads - 1) / kThreads;
  auto collect = [&](bool ties) {
    for (int w = tid; w < n_threads * per; w += kThreads) {
      const int v = sl.v0 + sh.threads[w % n_threads] + (w / n_threads) * kThreads;
      if (v >= sl.v1) continue;
      sl.each(v, [&](float x, int i) {
        if (x > tau || (ties && x == tau)) {
          const int c = atomicAdd(&sh.n_cand, 1);
          if (c < kCandidates) sh.cand[c] = Entry{x, i};
        }
      });
    }
    __syncthreads();
  };
  if (!many) collect(true);
  if (many || sh.n_cand > kCandidates) {
    __syncthreads();
    if (tid == 0) sh.n_cand = 0;
    __syncthreads();
    collect(false);
    if (sh.n_cand <= kCandidates - kMaxTop) {
      int have = sh.n_cand;
      __syncthreads();
      for (int base = sl.lo(); base < sl.hi() && have < want; base += kThreads) {
        const int i = base + tid;
        const bool hit = i < sl.hi() && Elem<T>::one(sl.row + i) == tau;
        const unsigned m = __ballot_sync(0xffffffffu, hit);
        if (lane == 0) sh.warp_count[warp] = __popc(m);
        __syncthreads();
        int at = have, all = 0;
        for (int w = 0; w < kWarps; ++w) {
          const int c = sh.warp_count[w];
          at += w < warp ? c : 0;
          all += c;
        }
        at += __popc(m & ((1u << lane) - 1));
        if (hit && at < want) sh.cand[at] = Entry{tau, i};
        have = min(want, have + all);
        __syncthreads();
      }
      if (tid == 0) sh.n_cand = max(have, sh.n_cand);
      __syncthreads();
    }
  }
  const int n = sh.n_cand;
  if (n <= kCandidates) {
    for (int c = tid; c < n; c += kThreads) {
      const Entry e = sh.cand[c];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += before(sh.cand[j], e);
      if (rank < want) sh.best[rank] = e;
    }
    __syncthreads();
    return want;
  }
  // More candidates than the buffer holds even so: one selection over the slice per entry.
  Entry last{INFINITY, -1};
  for (int s = 0; s < want; ++s) {
    Entry e{-INFINITY, 0x7fffffff};
    for (int v = sl.v0 + tid; v < sl.v1; v += kThreads)
      sl.each(v, [&](float x, int i) {
        const Entry c{x, i};
        if (before(last, c) && before(c, e)) e = c;
      });
    for (int o = 16; o > 0; o >>= 1) {
      const Entry c{__shfl_xor_sync(0xffffffffu, e.x, o), __shfl_xor_sync(0xffffffffu, e.i, o)};
      if (before(c, e)) e = c;
    }
    if (lane == 0) sh.red[warp] = e;
    __syncthreads();
    e = sh.red[0];
    for (int w = 1; w < kWarps; ++w)
      if (before(sh.red[w], e)) e = sh.red[w];
    if (tid == 0) sh.best[s] = e;
    last = e;
    __syncthreads();
  }
  return want;
}

template <class T>
__global__ void __launch_bounds__(kThreads, 2) token_logprobs_kernel(LogprobArgs a) {
  using E = Elem<T>;
  __shared__ __align__(16) Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int splits = static_cast<int>(cluster.num_blocks());
  const int split = static_cast<int>(cluster.block_rank());
  const int r = blockIdx.x / splits;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

  Slice<T> sl;
  sl.row = static_cast<const T*>(a.logits) + r * a.row_stride;
  sl.vocab = a.vocab;
  sl.off = static_cast<int>((reinterpret_cast<uintptr_t>(sl.row) & 15u) / sizeof(T));
  const int nvec = (a.vocab + sl.off + E::kPer - 1) / E::kPer;
  const int per_split = (nvec + splits - 1) / splits;
  sl.v0 = min(nvec, split * per_split);
  sl.v1 = min(nvec, sl.v0 + per_split);

  const int token = a.tokens != nullptr ? __ldg(a.tokens + r) : -1;
  const bool has_token = token >= 0 && token < a.vocab;
  const float xt = has_token ? E::one(sl.row + token) : INFINITY;

  Sums sums{kLowest, 0.f, 0.f};
  float mine = -INFINITY;  // largest element this thread read
  int above = 0;
  auto add_one = [&](float x) {
    mine = fmaxf(mine, x);
    above += x > xt;
    if (x > sums.ref + kGrowth) sums.move_to(x);
    const float t = max_nan(x - sums.ref, kFar) * kLog2e, e = fast_exp2(t);
    sums.s += e;
    sums.w = fmaf(e, t, sums.w);
  };
  // ends of the row that do not fill a vector, then the whole vectors
  int b0 = sl.v0, b1 = sl.v1;
  if (b0 < b1 && !sl.whole(b0)) {
    if (tid == 0) sl.each(b0, [&](float x, int) { add_one(x); });
  }
  if (b1 - 1 > b0 && !sl.whole(b1 - 1)) {
    if (tid == (b1 - 1 - b0) % kThreads) sl.each(b1 - 1, [&](float x, int) { add_one(x); });
    --b1;
  }
  const bool skip_first = b0 < b1 && !sl.whole(b0);
  for (int v = b0 + tid; v < b1; v += kBatch * kThreads) {
    uint4 u[kBatch];
    bool on[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int vk = v + k * kThreads;
      on[k] = vk < b1 && !(skip_first && vk == b0);
      if (on[k]) u[k] = sl.load(vk);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (!on[k]) continue;
      float2 x[E::kPer / 2];
      E::unpack(u[k], x);
      float mx = fmaxf(x[0].x, x[0].y);
#pragma unroll
      for (int j = 1; j < E::kPer / 2; ++j) mx = fmax3(mx, x[j].x, x[j].y);
      mine = fmaxf(mine, mx);
      if (mx > xt) {
#pragma unroll
        for (int j = 0; j < E::kPer / 2; ++j) above += (x[j].x > xt) + (x[j].y > xt);
      }
      if (mx > sums.ref + kGrowth) sums.move_to(mx);
      const float2 l2 = make_float2(kLog2e, kLog2e), nr = make_float2(-sums.ref, -sums.ref);
      float2 s2 = make_float2(0.f, 0.f), w2 = make_float2(0.f, 0.f);
#pragma unroll
      for (int j = 0; j < E::kPer / 2; ++j) {
        const float2 d = __fadd2_rn(x[j], nr);
        const float2 t = __fmul2_rn(make_float2(max_nan(d.x, kFar), max_nan(d.y, kFar)), l2);
        const float2 e = make_float2(fast_exp2(t.x), fast_exp2(t.y));
        s2 = __fadd2_rn(s2, e);
        w2 = __ffma2_rn(e, t, w2);
      }
      sums.s += s2.x + s2.y;
      sums.w += w2.x + w2.y;
    }
  }

  // the CTA's sums
  {
    Part p{sums, mine, above, 0};
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const Sums q{__shfl_xor_sync(0xffffffffu, p.sums.ref, o),
                   __shfl_xor_sync(0xffffffffu, p.sums.s, o),
                   __shfl_xor_sync(0xffffffffu, p.sums.w, o)};
      p.sums.merge(q);
      p.max = fmaxf(p.max, __shfl_xor_sync(0xffffffffu, p.max, o));
      p.above += __shfl_xor_sync(0xffffffffu, p.above, o);
    }
    if (lane == 0) sh.warp[warp] = p;
    __syncthreads();
    if (tid == 0) {
      for (int w = 1; w < kWarps; ++w) {
        p.sums.merge(sh.warp[w].sums);
        p.max = fmaxf(p.max, sh.warp[w].max);
        p.above += sh.warp[w].above;
      }
      sh.part = p;
    }
  }
  __syncthreads();
  int n_top = 0;
  if (a.top > 0) n_top = slice_top(sl, a.top, mine, sh);
  if (tid == 0) sh.part.top = n_top;
  __syncthreads();

  if (splits > 1) {
    cluster.sync();
    if (split == 0) {
      // every CTA's sums and entries into this one's shared memory
      if (tid == 0) {
        for (int c = 1; c < splits; ++c) {
          const Part q = *cluster.map_shared_rank(&sh.part, c);
          sh.part.sums.merge(q.sums);
          sh.part.max = fmaxf(sh.part.max, q.max);
          sh.part.above += q.above;
        }
      }
      if (a.top > 0) {
        const Entry none{-INFINITY, 0x7fffffff};
        for (int c = tid; c < splits * kMaxTop; c += kThreads) {
          const int from = c / kMaxTop, j = c % kMaxTop;
          const bool have = j < cluster.map_shared_rank(&sh.part, from)->top;
          sh.merged[c] = have ? cluster.map_shared_rank(sh.best, from)[j] : none;
        }
        __syncthreads();
        n_top = min(a.top, a.vocab);
        for (int c = tid; c < splits * kMaxTop; c += kThreads) {
          const Entry e = sh.merged[c];
          if (e.i == none.i) continue;
          int rank = 0;
          for (int j = 0; j < splits * kMaxTop; ++j) rank += before(sh.merged[j], e);
          if (rank < n_top) sh.cand[rank] = e;
        }
        __syncthreads();
        for (int c = tid; c < n_top; c += kThreads) sh.best[c] = sh.cand[c];
      }
      __syncthreads();
    }
    cluster.sync();  // nobody leaves while another CTA may read its shared memory
    if (split != 0) return;
  }

  const Part p = sh.part;
  const bool bad = isnan(p.sums.s) || p.max == INFINITY;  // NaN or +inf: no distribution
  const bool none = p.max == -INFINITY;  // every logit is -inf: nothing has probability
  Sums z = p.sums;
  z.move_to(p.max);
  const float log2z = log2f(z.s), ln_z = kLn2 * log2z;
  auto logprob = [&](float x) {
    return bad ? NAN : (none || x == -INFINITY) ? -INFINITY : (x - p.max) - ln_z;
  };
  if (tid == 0) {
    int bits = 0;
    if (bad) bits |= RB_EBIT_LOGITS;
    if (a.tokens != nullptr && !has_token && token != -1) bits |= RB_EBIT_TOKEN_ID;
    if (bits) raise_error(a.err, bits);
    if (a.logprobs != nullptr) a.logprobs[r] = has_token ? logprob(xt) : bad ? NAN : 0.f;
    if (a.ranks != nullptr) a.ranks[r] = has_token && !bad ? 1 + p.above : 0;
    if (a.entropy != nullptr)
      a.entropy[r] = bad ? NAN : none ? 0.f : fmaxf(0.f, kLn2 * (log2z - z.w / z.s));
  }
  if (tid < a.top) {
    const bool have = tid < n_top && !bad;
    a.top_ids[static_cast<long long>(r) * a.top + tid] = have ? sh.best[tid].i : -1;
    a.top_logprobs[static_cast<long long>(r) * a.top + tid] =
        have ? logprob(sh.best[tid].x) : bad ? NAN : -INFINITY;
  }
}

template <class T>
rb_status launch(const LogprobArgs& a, cudaStream_t s) {
  const int sms = max(1, device_sm_count());
  // CTAs per row: enough to give every SM two, each with at least 8 KiB of the row
  const long long row_bytes = static_cast<long long>(a.vocab) * sizeof(T);
  int splits = 1;
  while (splits < kMaxSplits && static_cast<long long>(a.rows) * splits < 2LL * sms &&
         row_bytes / (2 * splits) >= 8192)
    splits *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(a.rows) * splits));
  cfg.blockDim = dim3(kThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T>, a) != cudaSuccess) return RB_ERR_CUDA;
  note_launches(1);
  return RB_OK;
}

}  // namespace
}  // namespace rb

extern "C" rb_status rb_token_logprobs(int32_t num_rows, int32_t vocab_size, int64_t row_stride,
                                       int32_t logits_dtype, const void* d_logits,
                                       const int32_t* d_token_ids, int32_t top_k,
                                       float* d_logprobs, int32_t* d_ranks, float* d_entropy,
                                       int32_t* d_top_ids, float* d_top_logprobs,
                                       int32_t* d_error_word, void* stream) {
  rb::CallRange range_("rb_token_logprobs");
  using namespace rb;
  if (num_rows < 0 || vocab_size < 1 || top_k < 0 || row_stride < vocab_size)
    return RB_ERR_INVALID_ARG;
  if (top_k > kMaxTop || vocab_size > (1 << 30)) return RB_ERR_UNSUPPORTED;
  if (logits_dtype != RB_BF16 && logits_dtype != RB_FP16 && logits_dtype != RB_FP32)
    return RB_ERR_UNSUPPORTED;
  if (num_rows > 0x7fffffff / kMaxSplits) return RB_ERR_CAPACITY;
  if (num_rows == 0) return RB_OK;
  if (d_logits == nullptr || (top_k > 0 && (d_top_ids == nullptr || d_top_logprobs == nullptr)))
    return RB_ERR_INVALID_ARG;
  if (d_token_ids == nullptr && (d_logprobs != nullptr || d_ranks != nullptr))
    return RB_ERR_INVALID_ARG;
  const uintptr_t size = logits_dtype == RB_FP32 ? 4 : 2;
  if (reinterpret_cast<uintptr_t>(d_logits) % size != 0) return RB_ERR_INVALID_ARG;
  LogprobArgs a{d_logits, row_stride, d_token_ids, num_rows, vocab_size, top_k, d_logprobs,
                d_ranks, d_entropy, d_top_ids, d_top_logprobs, d_error_word};
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (logits_dtype == RB_FP32) return launch<float>(a, s);
  if (logits_dtype == RB_FP16) return launch<__half>(a, s);
  return launch<__nv_bfloat16>(a, s);
}
