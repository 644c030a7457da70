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
// The top k takes no part in that loop but maxima: each thread keeps the largest logit of each of
// up to eight segments of its share.  The k-th largest of 64 lane groups' maxima bounds the k-th
// largest logit from below; only segments whose maximum reaches it hold candidates, about k of
// the 8 per thread of a CTA, and those are read again (mostly from L2).
//
// Bound by HBM for many rows, by the chain of dependent steps (4 to 7 us) for few.  The next
// batch of 16-byte loads is issued before the current one is worked on, and the four CTAs of an SM
// of 256 threads (eight of 128 for short rows) hide each other's selection step.
#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "rb_internal.cuh"

namespace rb {
namespace {

namespace cg = cooperative_groups;

constexpr int kGroups = 64;       // lane groups whose maxima bound the k-th logit
constexpr int kSegments = 8;      // of a thread's share of the row, each with its own maximum
constexpr int kThreadsPerSm = 1024;
constexpr int kMaxTop = 32, kFew = 8;
constexpr int kMaxSplits = 8;     // CTAs of a cluster that share one row
constexpr int kCandidates = 1024;
constexpr long long kNarrowRow = 256 << 10;  // bytes up to which a row takes 128 threads
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// Differences to the reference are taken as at least kFar, so that masked (-inf) logits add
// 2^t t = 0 rather than 0 * inf.
constexpr float kFar = -1e30f;
constexpr float kGone = 1e4f;  // log2 units over which a sum that moves vanishes
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

// Elements of a 16-byte vector: their number, one of them, all as floats, all less a reference,
// the largest of several vectors' (NaN left out), and the vector of -inf.
template <class T>
struct Elem;
template <>
struct Elem<float> {
  static constexpr int kPer = 4, kBatch = 4;
  static constexpr uint32_t kNegInf = 0xff800000u;
  static __device__ __forceinline__ float one(const float* p) { return __ldg(p); }
  static __device__ __forceinline__ void unpack(const uint4& u, float2 (&x)[2]) {
    x[0] = make_float2(__uint_as_float(u.x), __uint_as_float(u.y));
    x[1] = make_float2(__uint_as_float(u.z), __uint_as_float(u.w));
  }
  static __device__ __forceinline__ void less(const uint4& u, float ref, float2 (&d)[2]) {
    unpack(u, d);
    const float2 nr = make_float2(-ref, -ref);
    d[0] = __fadd2_rn(d[0], nr);
    d[1] = __fadd2_rn(d[1], nr);
  }
  template <int N>
  static __device__ __forceinline__ float largest(const uint4 (&u)[N]) {
    float m[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int k = 0; k < N; ++k) {
      m[0] = fmax3(m[0], __uint_as_float(u[k].x), __uint_as_float(u[k].y));
      m[1] = fmax3(m[1], __uint_as_float(u[k].z), __uint_as_float(u[k].w));
    }
    return fmaxf(m[0], m[1]);
  }
};
// 16-bit types, two per word; less() is the mixed-precision subtraction, which converts as it
// subtracts (an unpacking instruction less per element).
// kBatch, vectors taken at a time with as many on their way.  4096 x 128000 bf16: 194 us, with 3
// vectors 196, with 2 215; 2047 x 100003 fp32: 147 us, with 2 vectors 165, with 6 (spills) 197.
template <class T, class Ops>
struct Elem16 {
  static constexpr int kPer = 8, kBatch = 4;
  static __device__ __forceinline__ float one(const T* p) {
    return Ops::two(__ldg(reinterpret_cast<const unsigned short*>(p))).x;
  }
  static __device__ __forceinline__ void unpack(const uint4& u, float2 (&x)[4]) {
    x[0] = Ops::two(u.x);
    x[1] = Ops::two(u.y);
    x[2] = Ops::two(u.z);
    x[3] = Ops::two(u.w);
  }
  static __device__ __forceinline__ void less(const uint4& u, float ref, float2 (&d)[4]) {
    d[0] = Ops::less(u.x, ref);
    d[1] = Ops::less(u.y, ref);
    d[2] = Ops::less(u.z, ref);
    d[3] = Ops::less(u.w, ref);
  }
  template <int N>
  static __device__ __forceinline__ float largest(const uint4 (&u)[N]) {
    uint32_t m[2] = {Ops::max2(u[0].x, u[0].y), Ops::max2(u[0].z, u[0].w)};
#pragma unroll
    for (int k = 1; k < N; ++k) {
      m[0] = Ops::max2(m[0], Ops::max2(u[k].x, u[k].y));
      m[1] = Ops::max2(m[1], Ops::max2(u[k].z, u[k].w));
    }
    const float2 x = Ops::two(Ops::max2(m[0], m[1]));
    return fmax3(x.x, x.y, -INFINITY);  // (both halves NaN: none)
  }
};
struct Bf16Ops {
  static __device__ __forceinline__ float2 two(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  static __device__ __forceinline__ float2 less(uint32_t w, float ref) {
    float2 d;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tsub.rn.f32.bf16 %0, l, %3;\n\t"
        "sub.rn.f32.bf16 %1, h, %3;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "r"(w), "f"(ref));
    return d;
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t y;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
  }
};
struct Fp16Ops {
  static __device__ __forceinline__ float2 two(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
  }
  static __device__ __forceinline__ float2 less(uint32_t w, float ref) {
    float2 d;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tsub.rn.f32.f16 %0, l, %3;\n\t"
        "sub.rn.f32.f16 %1, h, %3;\n\t}"
        : "=f"(d.x), "=f"(d.y)
        : "r"(w), "f"(ref));
    return d;
  }
  static __device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t y;
    asm("max.f16x2 %0, %1, %2;" : "=r"(y) : "r"(a), "r"(b));
    return y;
  }
};
template <>
struct Elem<__nv_bfloat16> : Elem16<__nv_bfloat16, Bf16Ops> {
  static constexpr uint32_t kNegInf = 0xff80ff80u;
};
template <>
struct Elem<__half> : Elem16<__half, Fp16Ops> {
  static constexpr uint32_t kNegInf = 0xfc00fc00u;
};

// s = sum 2^t, w = sum 2^t t with t = (x - ref) log2(e).
struct Sums {
  float ref, s, w;
  __device__ __forceinline__ void move_to(float to) {  // to >= ref
    if (s == 0.f) {
      w = 0.f;
    } else {
      // (beyond kGone f is 0; d itself would take d s past fp32's range)
      const float d = fminf((to - ref) * kLog2e, kGone), f = fast_exp2(-d);
      w = (w - d * s) * f;
      s *= f;
    }
    ref = to;
  }
};

struct Entry {
  float x;
  int i;
};
__device__ __forceinline__ bool before(const Entry& a, const Entry& b) {  // a ranks before b
  // no branch: it ranks hundreds of entries (3 x 306 bf16, top 20: 50 us with one, 12 without)
  return (a.x > b.x) | ((a.x == b.x) & (a.i < b.i));
}

struct Part {  // what one thread, warp, CTA or cluster found
  Sums sums;
  float max;
  int above;
};
__device__ __forceinline__ Part no_part() { return Part{Sums{kLowest, 0.f, 0.f}, -INFINITY, 0}; }

// Largest value of a warp's lanes (no NaN among them), by the integer order of the bits.
__device__ __forceinline__ float warp_max(float x) {
  const int b = __float_as_int(x);
  const int m = __reduce_max_sync(0xffffffffu, b >= 0 ? b : b ^ 0x7fffffff);
  return __int_as_float(m >= 0 ? m : m ^ 0x7fffffff);
}
// The parts of a warp's lanes as one, in every lane; kLanes: how many lanes in a row hold parts
// of their own (the others repeat them).  Each sum moves once, to the largest reference.
template <int kLanes>
__device__ __forceinline__ Part warp_merge(Part p) {
  p.sums.move_to(warp_max(p.sums.ref));
  p.max = warp_max(p.max);
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) {
    p.sums.s += __shfl_xor_sync(0xffffffffu, p.sums.s, o);
    p.sums.w += __shfl_xor_sync(0xffffffffu, p.sums.w, o);
    p.above += __shfl_xor_sync(0xffffffffu, p.above, o);
  }
  return p;
}

template <int kThreads>
struct Shared {
  static constexpr int kWarps = kThreads / 32;
  alignas(16) float group_max[kGroups];  // read four at a time
  Part warp[kWarps];
  Part part;
  Part parts[kMaxSplits];  // first CTA of a cluster: the others' sums
  float tau;
  int n_shares, n_cand;
  unsigned short shares[kThreads * kSegments];  // (thread, segment) pairs with candidates
  Entry cand[kCandidates];
  Entry red[kWarps];
  int warp_count[kWarps];
  Entry best[kMaxTop];
  Entry merged[kMaxSplits * kMaxTop];  // first CTA of a cluster: every CTA's entries
};

// One CTA's part of a row: 16-byte vectors [v0, v1) of the row's aligned vectors, of which
// [w0, w1) lie wholly in the row; the elements before and after those are taken one by one.
template <class T>
struct Slice {
  using E = Elem<T>;
  const T* row;
  int vocab, off, v0, v1, w0, w1;  // off: elements of vector 0 that lie before the row

  __device__ __forceinline__ int first(int v) const { return v * E::kPer - off; }
  __device__ __forceinline__ void bound() {
    w0 = v0;
    if (w0 < v1 && first(w0) < 0) ++w0;
    w1 = max(w0, first(v1) > vocab ? v1 - 1 : v1);
  }
  __device__ __forceinline__ uint4 load(int v) const {
    return __ldg(reinterpret_cast<const uint4*>(row + first(v)));
  }
  __device__ __forceinline__ int lo() const { return max(0, first(v0)); }
  __device__ __forceinline__ int hi() const { return min(vocab, first(v1)); }
  // The element outside the whole vectors that thread t takes (threads 0 to 31), or -1: those
  // before vector w0 and those from vector w1 on, at most 7 of each.
  __device__ __forceinline__ int edge(int t) const {
    const int lo_ = lo(), hi_ = hi(), front = min(hi_, first(w0)) - lo_;
    if (t < 16) return t < front ? lo_ + t : -1;
    const int i = max(lo_ + max(front, 0), first(w1)) + t - 16;
    return t < 32 && i < hi_ ? i : -1;
  }
};

// The top entries of a slice, in order, through emit(rank, entry); returns how many there are
// (min(k, elements)).  Thread t read vectors w0 + t + j * kThreads; segment g of its share are
// j in [g * per, (g + 1) * per), with maximum seg[g]; `edge_x` is its edge element (edge_i >= 0).
template <class T, int kThreads, class Emit>
__device__ __forceinline__ int slice_top(const Slice<T>& sl, int k, const float (&seg)[kSegments],
                                         int per, float edge_x, int edge_i, Shared<kThreads>& sh,
                                         Emit&& emit) {
  using E = Elem<T>;
  constexpr int kWarps = kThreads / 32, kPerGroup = kThreads / kGroups;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int want = min(k, max(0, sl.hi() - sl.lo()));
  if (want == 0) return 0;
  // The want-th largest group maximum: for few, one warp takes the largest that many times; for
  // many, every group's rank is counted, by all threads (8192 x 8000 bf16, top 5: 56 us against 58
  // by ranks; 2047 x 100003 fp32, top 20: 145 by ranks against 150).
  if (want <= kFew) {
    if (warp == 0) {
      float x = sh.group_max[lane], y = sh.group_max[lane + 32], m = 0.f;
      for (int i = 0; i < want; ++i) {
        m = warp_max(fmaxf(x, y));
        const unsigned who = __ballot_sync(0xffffffffu, x == m || y == m);
        if (lane == __ffs(who) - 1) {
          if (x == m) x = -INFINITY;
          else y = -INFINITY;
        }
      }
      if (lane == 0) sh.tau = m;
    }
  } else {
    const int g = tid / kPerGroup, share = tid % kPerGroup;
    const float x = sh.group_max[g];
    int rank = 0;
#pragma unroll
    for (int i = 0; i < kGroups / kPerGroup; i += 4) {
      const int j = share * (kGroups / kPerGroup) + i;
      const float4 o = *reinterpret_cast<const float4*>(sh.group_max + j);
      rank += (o.x > x || (o.x == x && j < g)) + (o.y > x || (o.y == x && j + 1 < g)) +
              (o.z > x || (o.z == x && j + 2 < g)) + (o.w > x || (o.w == x && j + 3 < g));
    }
#pragma unroll
    for (int o = 1; o < kPerGroup; o <<= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
    if (share == 0 && rank == want - 1) sh.tau = x;
  }
  __syncthreads();
  const float tau = sh.tau;  // at least `want` elements are >= tau (-inf: fewer groups had any)
  // Many elements equal to tau (masked logits above all): take those above it, then the first
  // equal ones in the order of their index.
  const bool many = tau == -INFINITY;
#pragma unroll
  for (int g = 0; g < kSegments; ++g)
    if (seg[g] > tau || (!many && seg[g] == tau))
      sh.shares[atomicAdd(&sh.n_shares, 1)] = static_cast<unsigned short>(tid + g * kThreads);
  __syncthreads();
  const int work = sh.n_shares * per;
  auto collect = [&](bool ties) {
    auto check = [&](float x, int i) {
      if (x > tau || (ties && x == tau)) {
        const int c = atomicAdd(&sh.n_cand, 1);
        if (c < kCandidates) sh.cand[c] = Entry{x, i};
      }
    };
    constexpr int kAhead = 4;
    for (int w0 = tid; w0 < work; w0 += kAhead * kThreads) {
      int v[kAhead];
      uint4 u[kAhead];
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int w = w0 + k * kThreads;
        v[k] = sl.w1;
        if (w < work) {
          const int q = sh.shares[w / per];
          v[k] = sl.w0 + q % kThreads + (q / kThreads * per + w % per) * kThreads;
        }
        if (v[k] < sl.w1) u[k] = sl.load(v[k]);
      }
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        if (v[k] >= sl.w1) continue;
        float2 x[E::kPer / 2];
        E::unpack(u[k], x);
#pragma unroll
        for (int j = 0; j < E::kPer / 2; ++j) {
          check(x[j].x, sl.first(v[k]) + 2 * j);
          check(x[j].y, sl.first(v[k]) + 2 * j + 1);
        }
      }
    }
    if (edge_i >= 0) check(edge_x, edge_i);
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
        const bool hit = i < sl.hi() && E::one(sl.row + i) == tau;
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
      if (rank < want) emit(rank, e);
    }
    return want;
  }
  // More candidates than the buffer holds even so: one selection over the slice per entry.
  Entry last{INFINITY, -1};
  for (int s = 0; s < want; ++s) {
    Entry e{-INFINITY, 0x7fffffff};
    for (int i = sl.lo() + tid; i < sl.hi(); i += kThreads) {
      const Entry c{E::one(sl.row + i), i};
      if (before(last, c) && before(c, e)) e = c;
    }
    for (int o = 16; o > 0; o >>= 1) {
      const Entry c{__shfl_xor_sync(0xffffffffu, e.x, o), __shfl_xor_sync(0xffffffffu, e.i, o)};
      if (before(c, e)) e = c;
    }
    if (lane == 0) sh.red[warp] = e;
    __syncthreads();
    e = sh.red[0];
    for (int w = 1; w < kWarps; ++w)
      if (before(sh.red[w], e)) e = sh.red[w];
    if (tid == 0) emit(s, e);
    last = e;
    __syncthreads();
  }
  return want;
}

// What a row's sums give: bad (NaN or +inf: no distribution), none (every logit is -inf: nothing
// has probability), ln Z relative to the maximum, and the entropy.
struct RowResult {
  bool bad, none;
  float max, ln_z, entropy;
  __device__ __forceinline__ explicit RowResult(const Part& p)
      : bad(isnan(p.sums.s) || p.max == INFINITY), none(p.max == -INFINITY), max(p.max) {
    Sums z = p.sums;
    z.move_to(p.max);
    const float log2z = log2f(z.s);
    ln_z = kLn2 * log2z;
    entropy = bad ? NAN : none ? 0.f : fmaxf(0.f, kLn2 * (log2z - z.w / z.s));
  }
  __device__ __forceinline__ float logprob(float x) const {
    return bad ? NAN : (none || x == -INFINITY) ? -INFINITY : (x - max) - ln_z;
  }
};

template <class T, int kBatch, int kThreads>
__global__ void __launch_bounds__(kThreads, kThreadsPerSm / kThreads)
    token_logprobs_kernel(LogprobArgs a) {
  using E = Elem<T>;
  constexpr int kWarps = kThreads / 32, kPerGroup = kThreads / kGroups;
  __shared__ Shared<kThreads> sh;
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
  sl.bound();

  const int stop = sl.w1;
  uint4 next[kBatch];
  auto fetch = [&](int v) {
#pragma unroll
    for (int k = 0; k < kBatch; ++k)
      if (v + k * kThreads < stop) next[k] = sl.load(v + k * kThreads);
  };
  fetch(sl.w0 + tid);
  const int token = a.tokens != nullptr ? __ldg(a.tokens + r) : -1;
  const bool has_token = token >= 0 && token < a.vocab;
  const float xt = has_token ? E::one(sl.row + token) : INFINITY;
  const int edge_i = tid < 32 ? sl.edge(tid) : -1;
  const float edge_x = edge_i >= 0 ? E::one(sl.row + edge_i) : -INFINITY;
  if (tid == 0) sh.n_shares = sh.n_cand = 0;

  // the thread's sums, even and odd elements apart, and largest element
  float ref = kLowest;
  float2 s2 = make_float2(0.f, 0.f), w2 = make_float2(0.f, 0.f);
  int above = 0;
  auto move_to = [&](float to) {
    Sums x{ref, s2.x, w2.x}, y{ref, s2.y, w2.y};
    x.move_to(to);
    y.move_to(to);
    s2 = make_float2(x.s, y.s);
    w2 = make_float2(x.w, y.w);
    ref = to;
  };
  float most = -INFINITY;
  if (edge_i >= 0) {
    most = edge_x;
    above = edge_x > xt;
    if (edge_x > ref + kGrowth) ref = edge_x;
    const float t = max_nan(edge_x - ref, kFar) * kLog2e;
    s2.x = fast_exp2(t);
    w2.x = s2.x * t;
  }
  // sums of one batch; kClamp: with -inf among the elements (2^t t would be 0 * inf)
  auto batch_sums = [&](const uint4 (&u)[kBatch], auto clamp, float2& bs, float2& bw) {
    constexpr bool kClamp = decltype(clamp)::value;
    const float2 l2 = make_float2(kLog2e, kLog2e);
    bs = bw = make_float2(0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      float2 d[E::kPer / 2];
      E::less(u[k], ref, d);
#pragma unroll
      for (int j = 0; j < E::kPer / 2; ++j) {
        if constexpr (kClamp) d[j] = make_float2(max_nan(d[j].x, kFar), max_nan(d[j].y, kFar));
        const float2 t = __fmul2_rn(d[j], l2);
        const float2 e = make_float2(fast_exp2(t.x), fast_exp2(t.y));
        bs = __fadd2_rn(bs, e);
        bw = __ffma2_rn(e, t, bw);
      }
    }
  };
  bool clamp = false;  // this thread's part of the row has -inf (or NaN) logits
  // a thread's share: `batches` rounds of kBatch vectors, cut into segments of `seg_batches`
  const int batches = (stop - sl.w0 + kBatch * kThreads - 1) / (kBatch * kThreads);
  const int seg_batches = max(1, (batches + kSegments - 1) / kSegments);
  float seg[kSegments];
#pragma unroll
  for (int g = 0; g < kSegments; ++g) seg[g] = -INFINITY;
  float top = -INFINITY;  // largest element of segment `at`, which ends before batch `end`
  int at = 0, end = seg_batches;
  // (one copy of the loop's code for all segments: with one for each, fetched anew, 4096 x 128000
  // bf16 took 214 us at its best batch, 4096 x 32000 71, now 194 and 60)
#pragma unroll 1
  for (int b = 0; b < batches; ++b) {
    const int v = sl.w0 + tid + b * (kBatch * kThreads);
    uint4 u[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      u[k] = next[k];
      if (v + k * kThreads >= stop) {  // past the end: -inf counts for nothing
        u[k] = make_uint4(E::kNegInf, E::kNegInf, E::kNegInf, E::kNegInf);
        clamp = true;
      }
    }
    fetch(v + kBatch * kThreads);
    const float mx = E::largest(u);
    top = fmaxf(top, mx);
    if (mx > xt) {
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        float2 x[E::kPer / 2];
        E::unpack(u[k], x);
#pragma unroll
        for (int j = 0; j < E::kPer / 2; ++j) above += (x[j].x > xt) + (x[j].y > xt);
      }
    }
    if (mx > ref + kGrowth) move_to(mx);
    float2 bs, bw;
    if (!clamp) {
      batch_sums(u, std::false_type{}, bs, bw);
      clamp = isnan(bw.x + bw.y);
    }
    if (clamp) batch_sums(u, std::true_type{}, bs, bw);
    s2 = __fadd2_rn(s2, bs);
    w2 = __fadd2_rn(w2, bw);
    if (b + 1 == end || b + 1 == batches) {
#pragma unroll
      for (int g = 0; g < kSegments; ++g) seg[g] = g == at ? top : seg[g];
      most = fmaxf(most, top);
      top = -INFINITY;
      ++at;
      end += seg_batches;
    }
  }
  Part mine{Sums{ref, s2.x + s2.y, w2.x + w2.y}, most, above};
  float group = mine.max;
#pragma unroll
  for (int o = 1; o < kPerGroup; o <<= 1)
    group = fmaxf(group, __shfl_xor_sync(0xffffffffu, group, o));
  if (tid % kPerGroup == 0) sh.group_max[tid / kPerGroup] = group;
  mine = warp_merge<32>(mine);
  if (lane == 0) sh.warp[warp] = mine;
  __syncthreads();
  Part p = warp_merge<kWarps>(sh.warp[lane % kWarps]);  // the CTA's sums, in every lane

  const long long top_row = static_cast<long long>(r) * a.top;
  int n_top = min(a.top, a.vocab);
  if (splits == 1) {
    const RowResult row(p);
    if (a.top > 0)
      slice_top(sl, a.top, seg, seg_batches * kBatch, edge_x, edge_i, sh,
                [&](int rank, const Entry& e) {
                  if (row.bad) return;
                  a.top_ids[top_row + rank] = e.i;
                  a.top_logprobs[top_row + rank] = row.logprob(e.x);
                });
  } else {
    cluster.sync();  // every CTA has started: its shared memory may be written
    Shared<kThreads>* first = cluster.map_shared_rank(&sh, 0);
    if (tid == 0) first->parts[split] = p;
    if (a.top > 0) {
      for (int c = tid; c < a.top; c += kThreads)
        first->merged[split * a.top + c] = Entry{-INFINITY, 0x7fffffff};
      __syncthreads();
      slice_top(sl, a.top, seg, seg_batches * kBatch, edge_x, edge_i, sh,
                [&](int rank, const Entry& e) { first->merged[split * a.top + rank] = e; });
    }
    cluster.sync();
    if (split != 0) return;
    p = warp_merge<kMaxSplits>(lane % kMaxSplits < splits ? sh.parts[lane % kMaxSplits]
                                                          : no_part());
    const RowResult row(p);
    if (warp == 0 && !row.bad) {  // merges the lists, lane l at the next entry of CTA l's
      const Entry end{-INFINITY, 0x7fffffff};
      auto entry = [&](int at) {
        return lane < splits && at < a.top ? sh.merged[lane * a.top + at] : end;
      };
      int at = 0;
      Entry e = entry(0);
      for (int k = 0; k < (a.top > 0 ? n_top : 0); ++k) {
        const float x = warp_max(e.x);
        const int i = __reduce_min_sync(0xffffffffu, e.x == x ? e.i : end.i);
        if (e.i == i && i != end.i) {
          a.top_ids[top_row + k] = i;
          a.top_logprobs[top_row + k] = row.logprob(e.x);
          e = entry(++at);
        }
      }
    }
  }
  if (warp != 0) return;
  const RowResult row(p);
  if (lane == 0) {
    int bits = 0;
    if (row.bad) bits |= RB_EBIT_LOGITS;
    if (a.tokens != nullptr && !has_token && token != -1) bits |= RB_EBIT_TOKEN_ID;
    if (bits) raise_error(a.err, bits);
    if (a.logprobs != nullptr) a.logprobs[r] = has_token ? row.logprob(xt) : row.bad ? NAN : 0.f;
    if (a.ranks != nullptr) a.ranks[r] = has_token && !row.bad ? 1 + p.above : 0;
    if (a.entropy != nullptr) a.entropy[r] = row.entropy;
  }
  if (row.bad) n_top = 0;
  if (lane >= n_top && lane < a.top) {  // entries there is no token for
    a.top_ids[top_row + lane] = -1;
    a.top_logprobs[top_row + lane] = row.bad ? NAN : -INFINITY;
  }
}

template <class T>
rb_status launch(const LogprobArgs& a, cudaStream_t s) {
  constexpr int kBatch = Elem<T>::kBatch;
  const int sms = max(1, device_sm_count());
  // CTAs per row: enough to give every SM two, each with at least 8 KiB of the row
  const long long row_bytes = static_cast<long long>(a.vocab) * sizeof(T);
  int splits = 1;
  while (splits < kMaxSplits && static_cast<long long>(a.rows) * splits < 2LL * sms &&
         row_bytes / (2 * splits) >= 8192)
    splits *= 2;
  // A short row's fixed steps weigh as much as its elements: twice as many CTAs per SM hide them
  // better.  16-bit logits, 256 -> 128 threads: 8192 x 8000 85 -> 56 us, 4096 x 32000 71 -> 60,
  // 4096 x 128000 194 -> 192; 6080 x 100000 fp32 384 -> 403.
  const bool narrow = splits == 1 && row_bytes <= kNarrowRow;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(static_cast<long long>(a.rows) * splits));
  cfg.blockDim = dim3(narrow ? 128 : 256);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = static_cast<unsigned>(splits);
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  void (*kernel)(LogprobArgs) = narrow ? token_logprobs_kernel<T, kBatch, 128>
                                       : token_logprobs_kernel<T, kBatch, 256>;
  if (cudaLaunchKernelEx(&cfg, kernel, a) != cudaSuccess) return RB_ERR_CUDA;
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
