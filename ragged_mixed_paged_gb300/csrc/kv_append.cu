// rb_kv_append, rb_kv4_append, rb_kv4_read: the step's queries and keys rotated by their
// positions, keys and values appended to the paged cache in 16 or in 4 bits, and rows of the 4-bit
// cache read back.
//
// Rotation: a pair (x, y) of a head becomes (x cos - y sin, y cos + x sin), the angles' cosines and
// sines taken from the caller's fp32 table; products and sums are rounded to fp32 one by one (no
// fused multiply-add), so that the result is the same whatever evaluates the formula.
#include <cfloat>

#include "kv4.cuh"

namespace rb {
namespace {

constexpr int kThreads = 128;

struct LayerScale {
  float scale, inverse;
};

struct AppendArgs {
  const __nv_bfloat16 *q, *k, *v;
  long long q_stride, k_stride, v_stride, q_out_stride;  // values between tokens
  const int32_t *positions, *slots;
  const float* table;
  __nv_bfloat16* q_out;
  void *k_cache, *v_cache;
  int32_t* err;
  long long num_slots;
  int tokens, nh, nkv, hd, rotary, max_position, interleaved, null_block;
  LayerScale k_scale, v_scale;
};

__device__ __forceinline__ float2 unpack2(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// (x, y) -> (x c - y s, y c + x s)
__device__ __forceinline__ void turn(float& x, float& y, float c, float s) {
  const float u = __fsub_rn(__fmul_rn(x, c), __fmul_rn(y, s));
  y = __fadd_rn(__fmul_rn(y, c), __fmul_rn(x, s));
  x = u;
}

// Sixteen values, as two 16-byte chunks: eight pairs, of adjacent values or of a value of each chunk.
__device__ __forceinline__ void turn16(uint4& a, uint4& b, const float (&c)[8], const float (&s)[8],
                                       bool interleaved) {
  uint32_t* pa = &a.x;
  uint32_t* pb = &b.x;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 x = unpack2(pa[i]), y = unpack2(pb[i]);
    if (interleaved) {
      turn(x.x, x.y, c[i], s[i]);
      turn(y.x, y.y, c[4 + i], s[4 + i]);
    } else {
      turn(x.x, y.x, c[2 * i], s[2 * i]);
      turn(x.y, y.y, c[2 * i + 1], s[2 * i + 1]);
    }
    pa[i] = pack_bf16x2(x.x, x.y);
    pb[i] = pack_bf16x2(y.x, y.y);
  }
}

// The larger magnitudes of two pairs of bf16 values; NaN where one is.
__device__ __forceinline__ uint32_t top2(uint32_t a, uint32_t b) {
  const __nv_bfloat162 m = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162*>(&a),
                                       *reinterpret_cast<const __nv_bfloat162*>(&b));
  return *reinterpret_cast<const uint32_t*>(&m);
}

// Codes and scale of sixteen bf16 values, written to their place; returns whether one of them was
// not finite (an infinity is held as the largest value, NaN as 0).  The largest magnitude is taken
// before the layer's scale divides the values: rounded quotients are in the values' order.
template <bool kValues>
__device__ __forceinline__ bool put_block(const uint4& a, const uint4& b, const LayerScale& by,
                                          uint8_t* cache, int slot, int head, int block, int nkv,
                                          int hd) {
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  constexpr uint32_t kAbs = 0x7fff7fffu;
  uint32_t m = w[0] & kAbs;
#pragma unroll
  for (int i = 1; i < 8; ++i) m = top2(m, w[i] & kAbs);
  m = top2(m, m << 16);  // (the high half)
  float top = __uint_as_float(m & 0xffff0000u);
  const bool odd = !(top <= FLT_MAX);
  float2 y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = unpack2(w[i]);
  if (by.scale != 1.f) {
    top = kv4::quotient(top, by.scale, by.inverse);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = kv4::quotient(y[i], by.scale, by.inverse);
  }
  if (!(top <= FLT_MAX)) {  // NaN, or beyond fp32 (the quotient of an infinity is NaN)
    top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      auto held = [&](float x, float q) {
        q = x != x ? 0.f : !(fabsf(q) <= FLT_MAX) ? copysignf(FLT_MAX, x) : q;
        top = fmaxf(top, fabsf(q));
        return q;
      };
      const float2 x = unpack2(w[i]);
      y[i] = make_float2(held(x.x, y[i].x), held(x.y, y[i].y));
    }
  }
  const uint32_t sb = kv4::scale_byte(__fdiv_rn(top, 6.f));
  const float s = kv4::scale_value(sb), r = sb != 0 ? __frcp_rn(s) : 0.f;  // (r = 0: codes of 0)
  uint32_t code[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = kv4::quotient(y[2 * i], s, r), u = kv4::quotient(y[2 * i + 1], s, r);
    code[i] = kv4::codes4(t.x, t.y, u.x, u.y);
  }
  const kv4::Place at = kv4::place<kValues>(slot, head, block, nkv, hd);
  *reinterpret_cast<uint2*>(cache + at.code) =
      make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
  cache[at.scale] = static_cast<uint8_t>(sb);
  return odd;
}

// One CTA per token.  A thread has one place in a head (the two chunks of a rotated or copied
// run of sixteen values), whose cosines and sines it holds, and takes every head of that place in
// turn, kBatch at a time so that their loads overlap; the first ones are on their way before
// position and slot are known.  The 4-bit cache's keys pass through shared memory as bf16,
// because the sixteen values that share a scale are not those of one thread's pairs.
//
// The 16-bit cache is HBM's: 16384 tokens of 32 + 16 heads of 128, 403 MB, take 66 us (seven CTAs an
// SM; six 70, five 77).  The 4-bit one has the codes' arithmetic as well, about 110 instructions a
// block, and the latency of a CTA's steps: slot, table, keys, codes (issue slots 0.63).  8192 tokens of
// 32 + 16 heads, 177 MB, take 38 us alone.  With the read of their rows behind them they take 51 with
// eight CTAs an SM (64 registers, two heads at a time), 58 with six and four heads at a time, and
// 68 where a thread codes its own halves of two blocks after a shuffle, without shared memory.
template <bool k4, int kBatch>
__global__ void __launch_bounds__(kThreads, k4 ? 8 : 7) append_kernel(const AppendArgs a) {
  extern __shared__ uint4 s_keys[];  // k4: the token's rotated keys
  const int t = blockIdx.x;
  const int per_head = a.hd / 16, lanes = kThreads / per_head;
  const int j = threadIdx.x % per_head, first = threadIdx.x / per_head;
  const int slot = __ldg(a.slots + t);
  const int pos = a.rotary > 0 ? __ldg(a.positions + t) : 0;
  // chunks of this thread's place in a head
  const bool turned = j < a.rotary / 16;
  const bool split = turned && !a.interleaved;
  const int ca = split ? j : 2 * j, cb = split ? j + a.rotary / 16 : 2 * j + 1;
  const int nq = a.q != nullptr ? a.nh : 0;
  const int heads = first < lanes ? nq + (k4 ? a.nkv : 2 * a.nkv) : 0;
  const __nv_bfloat16* q = a.q + t * a.q_stride;
  const __nv_bfloat16* k = a.k + t * a.k_stride;
  const __nv_bfloat16* v = a.v + t * a.v_stride;
  uint4 x[kBatch], y[kBatch];
  auto load = [&](int h0) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + i * lanes;
      if (h >= heads) break;
      const __nv_bfloat16* src = h < nq            ? q + static_cast<size_t>(h) * a.hd
                                 : h < nq + a.nkv ? k + static_cast<size_t>(h - nq) * a.hd
                                                  : v + static_cast<size_t>(h - nq - a.nkv) * a.hd;
      const uint4* p = reinterpret_cast<const uint4*>(src);
      x[i] = p[ca];
      y[i] = p[cb];
    }
  };
  load(first);
  // k4: the block of sixteen values that this thread quantises first, of K (below `blocks`) or V
  const int blocks = a.nkv * per_head;
  uint4 v0 = make_uint4(0u, 0u, 0u, 0u), v1 = v0;
  const int mine = static_cast<int>(threadIdx.x) - blocks;
  if (k4 && mine >= 0 && mine < blocks) {
    const uint4* p = reinterpret_cast<const uint4*>(v) + 2 * mine;
    v0 = p[0];
    v1 = p[1];
  }
  float c[8], s[8];
  if (a.rotary > 0) {
    if (pos < 0 || pos >= a.max_position) {  // the token is left out
      if (threadIdx.x == 0) raise_error(a.err, RB_EBIT_POSITION);
      return;
    }
    if (turned) {
      const float4* row =
          reinterpret_cast<const float4*>(a.table + static_cast<size_t>(pos) * a.rotary) + 2 * j;
      const float4 c0 = __ldg(row), c1 = __ldg(row + 1);
      const float4 s0 = __ldg(row + a.rotary / 8), s1 = __ldg(row + a.rotary / 8 + 1);
      c[0] = c0.x; c[1] = c0.y; c[2] = c0.z; c[3] = c0.w;
      c[4] = c1.x; c[5] = c1.y; c[6] = c1.z; c[7] = c1.w;
      s[0] = s0.x; s[1] = s0.y; s[2] = s0.z; s[3] = s0.w;
      s[4] = s1.x; s[5] = s1.y; s[6] = s1.z; s[7] = s1.w;
    }
  }
  const bool keep = slot >= 0 && slot < a.num_slots;
  if (slot >= a.num_slots && threadIdx.x == 0) raise_error(a.err, RB_EBIT_SLOT);
  __nv_bfloat16* q_out = a.q_out + t * a.q_out_stride;
  const size_t cache_row = static_cast<size_t>(keep ? slot : 0) * a.nkv * a.hd;
  __nv_bfloat16* k_out = k4 ? reinterpret_cast<__nv_bfloat16*>(s_keys)
                            : static_cast<__nv_bfloat16*>(a.k_cache) + cache_row;
  __nv_bfloat16* v_out = static_cast<__nv_bfloat16*>(a.v_cache) + cache_row;
  for (int h0 = first; h0 < heads; h0 += kBatch * lanes) {
    if (h0 != first) load(h0);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      const int h = h0 + i * lanes;
      if (h >= heads || (h >= nq && !keep)) break;
      __nv_bfloat16* dst;
      if (h < nq + a.nkv) {
        if (turned) turn16(x[i], y[i], c, s, a.interleaved != 0);
        dst = h < nq ? q_out + static_cast<size_t>(h) * a.hd
                     : k_out + static_cast<size_t>(h - nq) * a.hd;
      } else {
        dst = v_out + static_cast<size_t>(h - nq - a.nkv) * a.hd;
      }
      reinterpret_cast<uint4*>(dst)[ca] = x[i];
      reinterpret_cast<uint4*>(dst)[cb] = y[i];
    }
  }
  if constexpr (k4) {
    if (!keep) return;
    __syncthreads();
    bool odd = false;
    for (int i = threadIdx.x; i < 2 * blocks; i += kThreads) {
      if (i < blocks) {
        odd |= put_block<false>(s_keys[2 * i], s_keys[2 * i + 1], a.k_scale,
                                static_cast<uint8_t*>(a.k_cache), slot, i / per_head, i % per_head,
                                a.nkv, a.hd);
      } else {
        const int b = i - blocks;
        if (b != mine) {  // (not the one that is here already)
          const uint4* p = reinterpret_cast<const uint4*>(v) + 2 * b;
          v0 = p[0];
          v1 = p[1];
        }
        odd |= put_block<true>(v0, v1, a.v_scale, static_cast<uint8_t*>(a.v_cache), slot,
                               b / per_head, b % per_head, a.nkv, a.hd);
      }
    }
    if (odd && slot / kv4::kPage != a.null_block) raise_error(a.err, RB_EBIT_NOT_FINITE);
  }
}

template <bool k4>
rb_status launch_append(const AppendArgs& a, size_t smem, cudaStream_t s) {
  // heads that a thread takes: no more are loaded at a time, the fewer registers the more CTAs
  const int lanes = kThreads / (a.hd / 16);
  const int heads = (a.q != nullptr ? a.nh : 0) + (k4 ? a.nkv : 2 * a.nkv);
  if (heads <= lanes) append_kernel<k4, 1><<<a.tokens, kThreads, smem, s>>>(a);
  else if (k4 || heads <= 2 * lanes) append_kernel<k4, 2><<<a.tokens, kThreads, smem, s>>>(a);
  else append_kernel<false, 4><<<a.tokens, kThreads, smem, s>>>(a);
  if (last_launch_status() != RB_OK) return RB_ERR_CUDA;
  note_launches(1);
  return RB_OK;
}

// A thread per block of sixteen values of K and of V: nine bytes in, thirty-two out, in two stores
// that each fill half of their sectors.  8192 rows of 8 heads of 128, 43 MB, take 17 us cold (floor
// 6.3): three dependent loads (slot, codes, scale) and two divisions a block, and those stores.
template <bool kValues>
__device__ __forceinline__ void read_block(const uint8_t* cache, int slot, int head, int block,
                                           int nkv, int hd, float scale, uint4* dst) {
  const kv4::Place at = kv4::place<kValues>(slot, head, block, nkv, hd);
  const uint2 codes = *reinterpret_cast<const uint2*>(cache + at.code);
  const float s = kv4::scale_value(cache[at.scale]);
  uint32_t out[8];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h[4];
    kv4::values8(i == 0 ? codes.x : codes.y, h);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[k]));
      out[4 * i + k] = pack_bf16x2(f.x * s * scale, f.y * s * scale);
    }
  }
  dst[0] = make_uint4(out[0], out[1], out[2], out[3]);
  dst[1] = make_uint4(out[4], out[5], out[6], out[7]);
}

constexpr int kReadThreads = 256;

__global__ void __launch_bounds__(kReadThreads)
    read_kernel(int rows, int nkv, int hd, long long num_slots, const int32_t* slots,
                const uint8_t* kc, const uint8_t* vc, float k_scale, float v_scale, uint4* k_out,
                uint4* v_out, int32_t* err) {
  const int per_row = nkv * (hd / 16);
  const long long total = static_cast<long long>(rows) * per_row;
  const long long stride = static_cast<long long>(gridDim.x) * kReadThreads;
  for (long long i = static_cast<long long>(blockIdx.x) * kReadThreads + threadIdx.x; i < total;
       i += stride) {
    const int r = static_cast<int>(i / per_row), b = static_cast<int>(i - static_cast<long long>(r) * per_row);
    const int slot = __ldg(slots + r);
    if (slot < 0 || slot >= num_slots) {
      if (slot >= 0 && b == 0) raise_error(err, RB_EBIT_SLOT);
      k_out[2 * i] = k_out[2 * i + 1] = make_uint4(0u, 0u, 0u, 0u);
      v_out[2 * i] = v_out[2 * i + 1] = make_uint4(0u, 0u, 0u, 0u);
      continue;
    }
    const int head = b / (hd / 16), block = b - head * (hd / 16);
    read_block<false>(kc, slot, head, block, nkv, hd, k_scale, k_out + 2 * i);
    read_block<true>(vc, slot, head, block, nkv, hd, v_scale, v_out + 2 * i);
  }
}

// Host checks that both append entry points share; fills `a`.
rb_status append_setup(const rb_dims* dims, int32_t num_tokens_padded, const rb_rotation* rotation,
                       const int32_t* d_positions, const void* d_q, int64_t q_stride,
                       const void* d_k, int64_t k_stride, const void* d_v, int64_t v_stride,
                       const int32_t* d_slot_mapping, void* d_q_out, int64_t q_out_stride,
                       void* d_k_cache, void* d_v_cache, int32_t* d_error_word, AppendArgs* out) {
  if (dims == nullptr || num_tokens_padded < 0) return RB_ERR_INVALID_ARG;
  const rb_dims& d = *dims;
  if (d.block_size < 1 || d.num_kv_heads < 1 || d.num_q_heads < 1 || d.head_dim < 1 ||
      d.num_blocks < 1)
    return RB_ERR_INVALID_ARG;
  if (d.head_dim % 16 != 0 || d.head_dim > 2048) return RB_ERR_UNSUPPORTED;
  AppendArgs& a = *out;
  a = AppendArgs{};
  if (rotation != nullptr) {
    if (rotation->reserved != 0 || rotation->max_position < 1 || rotation->rotary_dim < 1 ||
        rotation->rotary_dim > d.head_dim || (rotation->interleaved & ~1) != 0)
      return RB_ERR_INVALID_ARG;
    if (rotation->rotary_dim % 16 != 0) return RB_ERR_UNSUPPORTED;
    a.rotary = rotation->rotary_dim;
    a.max_position = rotation->max_position;
    a.interleaved = rotation->interleaved;
    a.table = rotation->d_cos_sin;
  }
  if (num_tokens_padded == 0) return RB_OK;
  if (rotation != nullptr && (rotation->d_cos_sin == nullptr || d_positions == nullptr ||
                              !aligned16(rotation->d_cos_sin)))
    return RB_ERR_INVALID_ARG;
  if (d_k == nullptr || d_v == nullptr || d_slot_mapping == nullptr || d_k_cache == nullptr ||
      d_v_cache == nullptr || (d_q == nullptr) != (d_q_out == nullptr))
    return RB_ERR_INVALID_ARG;
  if (!aligned16(d_q) || !aligned16(d_k) || !aligned16(d_v) || !aligned16(d_q_out) ||
      !aligned16(d_k_cache) || !aligned16(d_v_cache))
    return RB_ERR_INVALID_ARG;
  const int64_t q_row = static_cast<int64_t>(d.num_q_heads) * d.head_dim;
  const int64_t kv_row = static_cast<int64_t>(d.num_kv_heads) * d.head_dim;
  if (k_stride < kv_row || v_stride < kv_row || k_stride % 8 != 0 || v_stride % 8 != 0)
    return RB_ERR_INVALID_ARG;
  if (d_q != nullptr &&
      (q_stride < q_row || q_out_stride < q_row || q_stride % 8 != 0 || q_out_stride % 8 != 0))
    return RB_ERR_INVALID_ARG;
  a.q = static_cast<const __nv_bfloat16*>(d_q);
  a.k = static_cast<const __nv_bfloat16*>(d_k);
  a.v = static_cast<const __nv_bfloat16*>(d_v);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_out_stride = q_out_stride;
  a.positions = d_positions;
  a.slots = d_slot_mapping;
  a.q_out = static_cast<__nv_bfloat16*>(d_q_out);
  a.k_cache = d_k_cache;
  a.v_cache = d_v_cache;
  a.err = d_error_word;
  a.num_slots = static_cast<long long>(d.num_blocks) * d.block_size;
  a.tokens = num_tokens_padded;
  a.nh = d.num_q_heads;
  a.nkv = d.num_kv_heads;
  a.hd = d.head_dim;
  a.null_block = d.null_block;
  return RB_OK;
}

// The 4-bit cache's own checks: its page, head and scale sizes, and slots that fit int32.
rb_status kv4_checks(const rb_dims& d, float k_scale, float v_scale) {
  if (d.block_size != kv4::kPage || (d.head_dim != 64 && d.head_dim != 128))
    return RB_ERR_UNSUPPORTED;
  if (static_cast<long long>(d.num_blocks) * d.block_size > 0x7fffffffLL) return RB_ERR_CAPACITY;
  return kv4::layer_scale_ok(k_scale) && kv4::layer_scale_ok(v_scale) ? RB_OK : RB_ERR_INVALID_ARG;
}

}  // namespace
}  // namespace rb

extern "C" rb_status rb_kv_append(const rb_dims* dims, int32_t num_tokens_padded,
                                  const rb_rotation* rotation, const int32_t* d_positions,
                                  const void* d_q, int64_t q_stride, const void* d_k,
                                  int64_t k_stride, const void* d_v, int64_t v_stride,
                                  const int32_t* d_slot_mapping, void* d_q_out,
                                  int64_t q_out_stride, void* d_k_cache, void* d_v_cache,
                                  int32_t* d_error_word, void* stream) {
  rb::CallRange range_("rb_kv_append");
  using namespace rb;
  AppendArgs a;
  const rb_status st = append_setup(dims, num_tokens_padded, rotation, d_positions, d_q, q_stride,
                                    d_k, k_stride, d_v, v_stride, d_slot_mapping, d_q_out,
                                    q_out_stride, d_k_cache, d_v_cache, d_error_word, &a);
  if (st != RB_OK || num_tokens_padded == 0) return st;
  return launch_append<false>(a, 0, static_cast<cudaStream_t>(stream));
}

extern "C" rb_status rb_kv4_append(const rb_dims* dims, int32_t num_tokens_padded,
                                   const rb_rotation* rotation, const int32_t* d_positions,
                                   const void* d_q, int64_t q_stride, const void* d_k,
                                   int64_t k_stride, const void* d_v, int64_t v_stride,
                                   const int32_t* d_slot_mapping, float k_scale, float v_scale,
                                   void* d_q_out, int64_t q_out_stride, void* d_k_cache,
                                   void* d_v_cache, int32_t* d_error_word, void* stream) {
  rb::CallRange range_("rb_kv4_append");
  using namespace rb;
  AppendArgs a;
  rb_status st = append_setup(dims, num_tokens_padded, rotation, d_positions, d_q, q_stride, d_k,
                              k_stride, d_v, v_stride, d_slot_mapping, d_q_out, q_out_stride,
                              d_k_cache, d_v_cache, d_error_word, &a);
  if (st != RB_OK) return st;
  st = kv4_checks(*dims, k_scale, v_scale);
  if (st != RB_OK || num_tokens_padded == 0) return st;
  a.k_scale = {k_scale, 1.f / k_scale};
  a.v_scale = {v_scale, 1.f / v_scale};
  const size_t smem = static_cast<size_t>(a.nkv) * a.hd * 2;
  if (smem > 48 * 1024) return RB_ERR_UNSUPPORTED;
  return launch_append<true>(a, smem, static_cast<cudaStream_t>(stream));
}

extern "C" rb_status rb_kv4_read(const rb_dims* dims, int32_t num_rows, const int32_t* d_slots,
                                 const void* d_k_cache, const void* d_v_cache, float k_scale,
                                 float v_scale, void* d_k_out, void* d_v_out,
                                 int32_t* d_error_word, void* stream) {
  rb::CallRange range_("rb_kv4_read");
  using namespace rb;
  if (dims == nullptr || num_rows < 0) return RB_ERR_INVALID_ARG;
  const rb_dims& d = *dims;
  if (d.num_kv_heads < 1 || d.head_dim < 1 || d.num_blocks < 1) return RB_ERR_INVALID_ARG;
  const rb_status st = kv4_checks(d, k_scale, v_scale);
  if (st != RB_OK || num_rows == 0) return st;
  if (d_slots == nullptr || d_k_cache == nullptr || d_v_cache == nullptr || d_k_out == nullptr ||
      d_v_out == nullptr || !aligned16(d_k_cache) || !aligned16(d_v_cache) ||
      !aligned16(d_k_out) || !aligned16(d_v_out))
    return RB_ERR_INVALID_ARG;
  const long long total = static_cast<long long>(num_rows) * d.num_kv_heads * (d.head_dim / 16);
  const long long want = (total + kReadThreads - 1) / kReadThreads;
  const long long most = 32LL * max(1, device_sm_count());
  read_kernel<<<static_cast<int>(want < most ? want : most), kReadThreads, 0,
                static_cast<cudaStream_t>(stream)>>>(
      num_rows, d.num_kv_heads, d.head_dim, static_cast<long long>(d.num_blocks) * d.block_size,
      d_slots, static_cast<const uint8_t*>(d_k_cache), static_cast<const uint8_t*>(d_v_cache),
      k_scale, v_scale, static_cast<uint4*>(d_k_out), static_cast<uint4*>(d_v_out), d_error_word);
  if (last_launch_status() != RB_OK) return RB_ERR_CUDA;
  note_launches(1);
  return RB_OK;
}
