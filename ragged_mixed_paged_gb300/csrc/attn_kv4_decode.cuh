// Split-KV decode warp of the attention over a 4-bit cache.  Not part of the C ABI.
//
// All decode requests' pages form one stream, of which every warp takes an equal part (Stream); a
// (request, kv head) whose pages end up with several warps is merged by the last one to finish.
// The contraction runs transposed, a 16-token page per MMA tile:
//   S^T[16 keys, 8 cols] = K[16, hd] . Q^T[hd, 8]     cols = (query token, head of the group)
//   O^T[hd, 8 cols]     += V^T[hd, 16] . P^T[16, 8]
// with mma.sync m16n8k16, fp16 in and fp32 accumulated.  Every value that the cache can hold is
// exact in fp16 (two bits of a code times four of a scale, between 2^-10 and 2880), so K and V enter
// the MMAs unrounded (times 2^-8, kScaleUnit); Q is divided by a power of two per column, which keeps
// its 8 bits.
//
// A page of one kv head is 9 hd contiguous bytes of K and as many of V.  A warp copies them to its
// own ring in shared memory with 16-byte cp.async, four pages ahead, and each lane then reads the
// bytes that are its MMA operands.  The MMA does not mind which 16 values of head_dim (K) or
// which dims and keys (V) a step takes, as long as both operands agree, so the order is chosen to
// make a lane's bytes neighbours.  With g = lane / 4, t = lane % 4:
//   K  rows g and g + 8 of the MMA are keys kg = 4 (g / 2) + g % 2 and kg + 2; lane (g, t) holds
//      values [t hd / 4, (t + 1) hd / 4) of both, and step s takes its s-th four values;
//   V  row g of step s is dim (hd / 8) g + 2 s and row g + 8 the next one; the lane holds the hd / 8
//      values of dims [(hd / 8) g, ...) of keys 4t .. 4t + 3, whose codes are paired by two
//      shifts and masks for a word of eight: neighbouring codes then belong to neighbouring keys.
// A lane so ends up with hd / 8 neighbouring values of two columns of the output.
//
// Two pages a step: their chains of MMAs and exponentials overlap, and the tests of a step are made
// once for both (256 decodes of 0.5 to 8 k 175 us with one, 171 with two, when that was the change).
// Where a segment (the pages of one head that a warp has) is odd, its last step takes one page twice,
// the second time unseen.
//
// What bounds it: instruction issue.  A page costs about 340 instructions a warp (hd 128), 310 cycles
// on the pipe of conversions, masks and shifts (64 conversions a lane, two cycles each); issue
// slots are at 0.63, the pipe at 0.54 (256 decodes of 4000 tokens: 224 us, 5.3 TB/s, 0.78 of the copy
// rate).  All 128 registers are taken; 44 bytes are spilled for heads of 128.
// A ring of 4, 5 or 6 pages makes no difference.
#pragma once

#include "attn_decode_warp.cuh"
#include "kv4.cuh"

namespace rb {
namespace attn {

// The kernel's arguments: the ordinary ones, whose scale_log2 includes k_scale, and the cache.
struct Kv4Args {
  AttnArgs a;
  const uint8_t *k, *v;
  float v_scale;
};

// Probabilities are held in fp16 for P V.  A reference is set so that the largest one is 2^kPShift
// when it is taken: smaller ones keep their 11 bits down to 2^-20 of the largest and vanish below
// 2^-31 of it, so that even 2^17 vanishing keys are 2^-14 of the sum.
constexpr float kPShift = 6.f;

namespace kv4d {

// 2^-e and 2^e for a column (row) whose largest |q| is `top`: q 2^-e is below 2 and exact in fp16
// (values below 2^-14 of it to 2^-25 of it).
__device__ __forceinline__ void power_of(float top, float* down, float* up) {
  const uint32_t e = min(max(__float_as_uint(top) >> 23, 1u), 253u);
  const bool odd = !(top < INFINITY);
  *down = odd ? 1.f : __uint_as_float((254u - e) << 23);
  *up = odd ? 1.f : __uint_as_float(e << 23);
}

// What turns a column's (row's) raw products into log2 units: 2^e times the call's factor, kept
// above 0 and finite, so that neither a masked score (-inf) nor a raw score of 0 becomes NaN.  Raw
// products are below 2^13: scores under the lower bound are 0 to within 2^-87.  They are multiples of
// 2^-42 (of q's 2^-24 and the cache's 2^-18): above the upper one any two that differ are 2^58 apart.
// kNoReference is the offset of a column that has no reference yet: it puts any product far above one.
__device__ __forceinline__ float score_scale(float up, float unit) {
  return fminf(fmaxf(up * unit, 0x1p-100f), 0x1p100f);
}
constexpr float kNoReference = 0x1p120f;

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&a),
                            *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Scale bytes of `w` as a half2 (kv4::scale_value of each), times 2^-8: a byte's seven bits lie in a
// half's fields as they are, the biases being 7 and 15.  A product with a code stays exact, down to
// 2^-18 among fp16's subnormals.  kSelect names the bytes (byte_perm with 0: 0x4140 bytes 0 and
// 1, 0x4040 byte 0 twice).
constexpr float kScaleUnit = 256.f;
template <int kSelect>
__device__ __forceinline__ uint32_t scales2(uint32_t w) {
  return __byte_perm(w & 0x7f7f7f7fu, 0, kSelect) << 7;
}

// D = A B + C
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1, float c0, float c1,
                                        float c2, float c3) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// Geometry of a warp's ring: pages as they lie in the cache, but for the order of rows, which keeps the
// lanes' reads free of bank conflicts and the places of a lane's copies a constant apart.
//   K: the lanes' first rows, in order of g, then their second ones: lane's bytes at lane x hd / 8
//   V: row 4t + i at row t % 2 + 2i of half t / 2, the halves 32 or 64 bytes apart
template <int HD>
struct Ring {
  static constexpr int kStages = 6;              // pages; a step takes two
  static constexpr int kRow = HD / 2;            // bytes of codes of a row
  static constexpr int kBytes = 9 * HD;          // K or V of a page in the cache
  static constexpr int kVHalf = 8 * kRow + (HD == 128 ? 32 : 64);
  static constexpr int kV = kBytes;              // V codes, K codes being at 0
  static constexpr int kKScales = 16 * kRow, kVScales = kV + 2 * kVHalf;
  static constexpr int kStageBytes = kVScales + HD;
  static constexpr int kWarpBytes = kStages * kStageBytes;
  static constexpr int kCopies = 16 * kRow / 512;  // of 16 bytes a lane: K (V) codes
  static constexpr int kScaleLanes = HD / 16;      // lanes that copy the scales
};

template <int kTo, int kFrom>
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;" ::"r"(dst), "l"(src), "n"(kTo),
               "n"(kFrom)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {  // all but the last N groups have landed
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Words of a ring at a shared-memory address and a constant distance.
template <int kAt, int N>
__device__ __forceinline__ void read_words(uint32_t (&r)[N], uint32_t at) {
  if constexpr (N == 4)
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4 + %5];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(at), "n"(kAt));
  else if constexpr (N == 2)
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2 + %3];"
                 : "=r"(r[0]), "=r"(r[1])
                 : "r"(at), "n"(kAt));
  else
    asm volatile("ld.shared.u32 %0, [%1 + %2];" : "=r"(r[0]) : "r"(at), "n"(kAt));
}
template <int kAt, int kBytes>
__device__ __forceinline__ uint32_t read_scales(uint32_t at) {
  uint16_t v;
  if constexpr (kBytes == 2)
    asm volatile("ld.shared.u16 %0, [%1 + %2];" : "=h"(v) : "r"(at), "n"(kAt));
  else
    asm volatile("ld.shared.u8 %0, [%1 + %2];" : "=h"(v) : "r"(at), "n"(kAt));
  return v;
}

// A lane's places in a stage: its K codes and scales, its V codes and scales.
template <int HD>
struct Places {
  int k, k_scale, v, v_scale;
  __device__ explicit Places(int lane) {
    const int g = lane >> 2, t = lane & 3, key_g = 4 * (g >> 1) + (g & 1);
    using R = Ring<HD>;
    k = lane * (HD / 8);
    k_scale = R::kKScales + key_g * (HD / 16) + t * (HD / 64);
    v = R::kV + (t >> 1) * R::kVHalf + (t & 1) * R::kRow + g * (HD / 16);
    v_scale = R::kVScales + g * (HD / 8) / 16 * 16 + 4 * t;
  }
};

// S^T of the page at `stage` (over kScaleUnit): two chains of MMAs.
template <int HD>
__device__ __forceinline__ void scores(uint32_t stage, const Places<HD>& at,
                                       const uint32_t (&bq)[HD / 16][2], float (&s)[4]) {
  uint32_t c0[HD / 32], c1[HD / 32];
  read_words<0>(c0, stage + at.k);
  read_words<8 * (HD / 2)>(c1, stage + at.k);
  const uint32_t w0 = read_scales<0, HD / 64>(stage + at.k_scale);
  const uint32_t w1 = read_scales<2 * (HD / 16), HD / 64>(stage + at.k_scale);
  // (a lane's HD / 4 values are one block of 16 for HD 64, two for 128)
  const uint32_t m00 = scales2<0x4040>(w0), m01 = HD == 128 ? scales2<0x4141>(w0) : 0u;
  const uint32_t m10 = scales2<0x4040>(w1), m11 = HD == 128 ? scales2<0x4141>(w1) : 0u;
  float s2[4];
#pragma unroll
  for (int w = 0; w < HD / 32; ++w) {
    const uint32_t m0 = w < 2 ? m00 : m01, m1 = w < 2 ? m10 : m11;
    uint32_t x[4], y[4];
    kv4::values8(c0[w], x);
    kv4::values8(c1[w], y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = hmul2(x[i], m0);
      y[i] = hmul2(y[i], m1);
    }
    if (w == 0) {
      mma_f16(s, x[0], y[0], x[1], y[1], bq[0][0], bq[0][1], 0.f, 0.f, 0.f, 0.f);
      mma_f16(s2, x[2], y[2], x[3], y[3], bq[1][0], bq[1][1], 0.f, 0.f, 0.f, 0.f);
    } else {
      mma_f16(s, x[0], y[0], x[1], y[1], bq[2 * w][0], bq[2 * w][1], s[0], s[1], s[2], s[3]);
      mma_f16(s2, x[2], y[2], x[3], y[3], bq[2 * w + 1][0], bq[2 * w + 1][1], s2[0], s2[1], s2[2],
              s2[3]);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] += s2[i];
}

// O^T += V^T P^T of the page at `stage` (V over kScaleUnit).
template <int HD>
__device__ __forceinline__ void add_values(uint32_t stage, const Places<HD>& at, uint32_t pb0,
                                           uint32_t pb1, float (&acc)[HD / 16][4]) {
  uint32_t sv[1], c[4][HD / 64];
  read_words<0>(sv, stage + at.v_scale);
  read_words<0>(c[0], stage + at.v);
  read_words<2 * (HD / 2)>(c[1], stage + at.v);
  read_words<4 * (HD / 2)>(c[2], stage + at.v);
  read_words<6 * (HD / 2)>(c[3], stage + at.v);
  const uint32_t s01 = scales2<0x4140>(sv[0]), s23 = scales2<0x4342>(sv[0]);
#pragma unroll
  for (int w = 0; w < HD / 64; ++w) {
    // even and odd dims of a word, the first key of a pair in the low half of each byte
    auto even = [](uint32_t x, uint32_t y) { return (x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u); };
    auto odd = [](uint32_t x, uint32_t y) { return ((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u); };
    uint32_t e01[4], o01[4], e23[4], o23[4];
    kv4::values8(even(c[0][w], c[1][w]), e01);
    kv4::values8(odd(c[0][w], c[1][w]), o01);
    kv4::values8(even(c[2][w], c[3][w]), e23);
    kv4::values8(odd(c[2][w], c[3][w]), o23);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float(&d)[4] = acc[4 * w + i];
      mma_f16(d, hmul2(e01[i], s01), hmul2(o01[i], s01), hmul2(e23[i], s23), hmul2(o23[i], s23),
              pb0, pb1, d[0], d[1], d[2], d[3]);
    }
  }
}

}  // namespace kv4d

// Log-sum-exp merge of the pieces of one (request, kv head) by one warp, kLanes lanes per column,
// each lane owning that part of head_dim.  Piece 0 is the last one of its warp, the others are the
// first of theirs.  Partials of other SMs are read through L2, 16 loads in flight.  They are sums of
// weights of up to 2^(kPShift + 8) over V without its scale `v_unit`, which would take them out of
// fp32's range before the division.
template <int HD, int kLanes>
__device__ __forceinline__ void merge_pieces(const AttnArgs& a, int w0, int n, int h, int t0,
                                             int cols, float v_unit) {
  constexpr int kPer = HD / kLanes, kVec = kPer / 4, kBatch = 16 / kVec;
  const int lane = threadIdx.x & 31;
  const int col = lane / kLanes, part = lane % kLanes;
  const bool active = col < cols;
  const int c = active ? col : 0;
  auto slot = [&](int i) { return static_cast<size_t>(i == 0 ? 2 * w0 + 1 : 2 * (w0 + i)); };
  float mx = -INFINITY;
#pragma unroll 2
  for (int i = part; i < n; i += kLanes)
    mx = fmaxf(mx, __ldcg(&a.part_ml[slot(i) * kMaxCols + c].x));
#pragma unroll
  for (int o = 1; o < kLanes; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  if (mx == -INFINITY) mx = 0.f;
  float acc[kPer], sum = 0.f;
#pragma unroll
  for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
#pragma unroll 1
  for (int i0 = 0; i0 < n; i0 += kBatch) {
    float2 ml[kBatch];
    float4 x[kBatch][kVec];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const size_t u = slot(min(i0 + k, n - 1)) * kMaxCols + c;
      ml[k] = __ldcg(a.part_ml + u);
#pragma unroll
      for (int v = 0; v < kVec; ++v)
        x[k][v] = __ldcg(reinterpret_cast<const float4*>(a.part_o + u * HD + part * kPer) + v);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if (i0 + k >= n) break;
      const float w = fast_exp2(ml[k].x - mx);
      sum += w * ml[k].y;
#pragma unroll
      for (int v = 0; v < kVec; ++v) {
        acc[4 * v + 0] += w * x[k][v].x;
        acc[4 * v + 1] += w * x[k][v].y;
        acc[4 * v + 2] += w * x[k][v].z;
        acc[4 * v + 3] += w * x[k][v].w;
      }
    }
  }
  if (!active) return;
  const int j = col / a.group, hh = col - j * a.group;
  const float inv = v_unit / sum;  // (a row of nothing but -inf: 0 / 0)
  uint2* dst = reinterpret_cast<uint2*>(
      a.out + (static_cast<size_t>(t0 + j) * a.nh + h * a.group + hh) * HD + part * kPer);
#pragma unroll
  for (int v = 0; v < kVec; ++v)
    dst[v] = make_uint2(pack_bf16x2(acc[4 * v + 0] * inv, acc[4 * v + 1] * inv),
                        pack_bf16x2(acc[4 * v + 2] * inv, acc[4 * v + 3] * inv));
}

// What the decode phase reads, as one stream of pages: requests in order, of each the kv heads, of
// each the pages.  a.dec_off[r] counts the pages of one head of the decode requests before r.  Warp w
// of W takes pages [T w / W, T (w + 1) / W) of the T, so all end together, and a warp's copies go
// on across the ends of heads and requests.
struct Stream {
  long long total;
  int warps;
  __device__ Stream(const AttnArgs& a)
      : total(static_cast<long long>(a.dec_off[a.R]) * a.nkv), warps(a.header[kHNumDecodeUnits]) {}
  __device__ long long begin(int w) const { return total * w / warps; }
  __device__ int warp_of(long long x) const {
    return static_cast<int>(((x + 1) * warps - 1) / total);
  }
};
// A place in the stream.
struct Place {
  int r, h, page, pages;
  __device__ Place(const AttnArgs& a, long long x) {
    r = warp_upper_bound_i32(a.dec_off, a.R + 1, static_cast<int>(x / a.nkv)) - 1;
    const int off = a.dec_off[r];
    pages = a.dec_off[r + 1] - off;
    const long long local = x - static_cast<long long>(off) * a.nkv;
    h = static_cast<int>(local / pages);
    page = static_cast<int>(local - static_cast<long long>(h) * pages);
  }
  __device__ void head_end(const AttnArgs& a, bool more) {  // after the head's last page
    page = 0;
    if (++h < a.nkv || !more) return;
    h = 0;
    int off = a.dec_off[r + 1], next;
    do {  // (more: there is a request with pages)
      ++r;
      next = a.dec_off[r + 1];
    } while (next == off);
    pages = next - off;
  }
};

// One decode warp, w of the stream's; `ring` is its kv4d::Ring in shared memory.
template <int HD>
__device__ void decode_warp_kv4(const Kv4Args& g4, uint8_t* ring, int w) {
  using namespace kv4d;
  using R = Ring<HD>;
  const AttnArgs& a = g4.a;
  constexpr int kKS = HD / 16, kPer = HD / 8;  // MMA steps; output values of a lane and column
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const Stream stream(a);
  if (w >= stream.warps) return;
  const long long x0 = stream.begin(w);
  const int n = static_cast<int>(stream.begin(w + 1) - x0);
  Place at(a, x0);  // of the next page to compute

  // Copies: page ids of up to 32 pages of one head a window, one per lane, the next one prefetched.
  Place from = at;  // of the first page after the prefetched window
  int left = n;
  bool bad = false;
  struct Window {
    int id, n, h;
  };
  auto window = [&]() {
    Window x{0, min(32, min(from.pages - from.page, left)), from.h};
    if (lane < x.n) {
      x.id = kernel_page(a.block_table + static_cast<size_t>(from.r) * a.MB, from.page + lane,
                         a.ratio, a.num_blocks, a.null_block);
      if (x.id < 0) {
        bad = true;
        x.id = a.null_block;
      }
    }
    left -= x.n;
    from.page += x.n;
    if (from.page == from.pages) from.head_end(a, left > 0);
    return x;
  };
  Window now = window(), next = window();
  int pos = 0, to_copy = n;
  const uint32_t ring_at = smem_u32(ring), ring_end = ring_at + R::kWarpBytes;
  uint32_t copy_to = ring_at;
  const uint32_t page_stride = static_cast<uint32_t>(a.nkv) * R::kBytes;
  const uint8_t *k_src, *v_src;  // this lane's chunks of page 0 of the window's head
  auto sources = [&] {
    k_src = g4.k + now.h * R::kBytes + lane * 16;
    v_src = g4.v + now.h * R::kBytes + lane * 16;
  };
  sources();
  // where this lane's first chunks of codes go in a stage (its second ones are rows 8 further on)
  const int chunks = HD / 32, row = lane / chunks, in_row = lane % chunks * 16;
  const int k_to = ((row >> 2) * 2 + (row & 1) + 8 * (row >> 1 & 1)) * R::kRow + in_row;
  const int v_to = R::kV + (row >> 3) * R::kVHalf + ((row >> 2 & 1) + 2 * (row & 3)) * R::kRow + in_row;
  auto copy = [&]() {  // the next page; past the last one an empty group
    if (to_copy > 0) {
      --to_copy;
      if (pos == now.n) {
        now = next;
        pos = 0;
        sources();
        next = window();
      }
      const uint32_t id = __shfl_sync(0xffffffffu, now.id, pos++);
      const uint8_t* ks = k_src + static_cast<uint64_t>(id) * page_stride;
      const uint8_t* vs = v_src + static_cast<uint64_t>(id) * page_stride;
      copy16<0, 0>(copy_to + k_to, ks);
      copy16<0, 0>(copy_to + v_to, vs);
      if constexpr (R::kCopies == 2) {
        copy16<4 * R::kRow, 512>(copy_to + k_to, ks);
        copy16<R::kVHalf, 512>(copy_to + v_to, vs);
      }
      if (lane < R::kScaleLanes) {
        copy16<R::kKScales, 16 * R::kRow>(copy_to + lane * 16, ks);
        copy16<R::kVScales, 16 * R::kRow>(copy_to + lane * 16, vs);
      }
      copy_to += R::kStageBytes;
      if (copy_to == ring_end) copy_to = ring_at;
    }
    copies_commit();
  };
  constexpr int kAhead = R::kStages - 2;  // pages copied beyond those that are done with
#pragma unroll 1
  for (int i = 0; i < kAhead; ++i) copy();

  const int key_g = 4 * (g >> 1) + (g & 1);  // key of the lane's first K row
  const Places<HD> places(lane);
  uint32_t stage = ring_at;
  for (int done = 0; done < n;) {  // segments: pages of one (request, kv head)
    const int r = at.r, h = at.h, first = at.page, pages = at.pages;
    const int seg = min(pages - first, n - done);
    done += seg;
    at.page += seg;
    if (at.page == pages) at.head_end(a, done < n);
    const int t0 = a.qsl[r], q = a.qsl[r + 1] - t0, c = a.seq_lens[r] - q, cols = q * a.group;
    // Q^T fragments: column g, values [t hd / 4, (t + 1) hd / 4) over 2^e
    uint32_t bq[kKS][2];
    float up;
    {
      const bool valid = g < cols;
      const int j = valid ? g / a.group : 0;
      const int hh = valid ? g - j * a.group : 0;
      const uint4* qp = reinterpret_cast<const uint4*>(
          a.q + (static_cast<size_t>(t0 + j) * a.nh + h * a.group + hh) * HD + t * (HD / 4));
      uint4 word[HD / 32];
#pragma unroll
      for (int i = 0; i < HD / 32; ++i) word[i] = valid ? __ldg(qp + i) : make_uint4(0u, 0u, 0u, 0u);
      const uint32_t* qw = reinterpret_cast<const uint32_t*>(word);
      float top = 0.f;
#pragma unroll
      for (int i = 0; i < HD / 8; ++i)
        top = fmax3(top, fabsf(__uint_as_float(qw[i] << 16)),
                    fabsf(__uint_as_float(qw[i] & 0xffff0000u)));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      float down;
      power_of(top, &down, &up);
#pragma unroll
      for (int i = 0; i < HD / 8; ++i)
        bq[i / 2][i % 2] = pack_f16x2(__uint_as_float(qw[i] << 16) * down,
                                      __uint_as_float(qw[i] & 0xffff0000u) * down);
    }
    // the lane's columns of S^T: their scales and their last visible key
    const int c0 = 2 * t, c1 = c0 + 1;
    const float unit = a.scale_log2 * kScaleUnit;
    const float sc0 = score_scale(__shfl_sync(0xffffffffu, up, 4 * c0), unit);
    const float sc1 = score_scale(__shfl_sync(0xffffffffu, up, 4 * c1), unit);
    const int lim0 = c0 < cols ? c + c0 / a.group : c;
    const int lim1 = c1 < cols ? c + c1 / a.group : c;
    // Exponents are taken against a reference, one of the raw products, that moves only when one
    // exceeds it by more than kGrowth (log2 units), so that P stays below 2^(kPShift + kGrowth).  It
    // is taken off the raw products, so that their differences keep their bits however large the scores
    // are; an offset in log2 units gives infinite weights from scores of 2^23 on.  (256 decodes 169 us,
    // 167 with such an offset; the raw difference only for segments with a large factor is no faster.)
    constexpr float kGrowth = 8.f;
    const float2 sc = make_float2(sc0, sc1);
    float2 off = make_float2(kNoReference, kNoReference), l = make_float2(0.f, 0.f);  // (-reference)
    float acc[kKS][4];
#pragma unroll
    for (int mt = 0; mt < kKS; ++mt) acc[mt][0] = acc[mt][1] = acc[mt][2] = acc[mt][3] = 0.f;
    // pages whose keys every column sees (the columns' last keys are c and more)
    const int whole = min(first + seg, (c + 1) / kPage);
    // Two pages a step; the last one's second page may be missing: it is the first one again, unseen.
#pragma unroll 1
    for (int page = first; page < first + seg; page += 2) {
      copies_wait<kAhead - 2>();
      __syncwarp();  // both have landed for every lane, and every lane is done with those before
      uint32_t other = stage + R::kStageBytes;
      if (other == ring_end) other = ring_at;
      const bool both = page + 1 < first + seg;
      if (!both) other = stage;
      float s[4], u[4];
      scores<HD>(stage, places, bq, s);
      scores<HD>(other, places, bq, u);
      if (page + 1 >= whole) {
        const int key = page * kPage + key_g;
        s[0] = key <= lim0 ? s[0] : -INFINITY;
        s[1] = key <= lim1 ? s[1] : -INFINITY;
        s[2] = key + 2 <= lim0 ? s[2] : -INFINITY;
        s[3] = key + 2 <= lim1 ? s[3] : -INFINITY;
        const int next = both ? key + kPage : 0x7ffffff0;
        u[0] = next <= lim0 ? u[0] : -INFINITY;
        u[1] = next <= lim1 ? u[1] : -INFINITY;
        u[2] = next + 2 <= lim0 ? u[2] : -INFINITY;
        u[3] = next + 2 <= lim1 ? u[3] : -INFINITY;
      }
      float g0 = fmax3(fmaxf(s[0], s[2]), u[0], u[2]), g1 = fmax3(fmaxf(s[1], s[3]), u[1], u[3]);
      const float2 above = __fmul2_rn(__fadd2_rn(make_float2(g0, g1), off), sc);
      if (__any_sync(0xffffffffu, above.x > kGrowth || above.y > kGrowth)) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          g0 = fmaxf(g0, __shfl_xor_sync(0xffffffffu, g0, o));
          g1 = fmaxf(g1, __shfl_xor_sync(0xffffffffu, g1, o));
        }
        const float2 old = off;  // (a column keeps its own, whatever the others do)
        if ((g0 + old.x) * sc0 > kGrowth) off.x = -g0;
        if ((g1 + old.y) * sc1 > kGrowth) off.y = -g1;
        const float al0 = fast_exp2((off.x - old.x) * sc0), al1 = fast_exp2((off.y - old.y) * sc1);
        l = __fmul2_rn(l, make_float2(al0, al1));
#pragma unroll
        for (int mt = 0; mt < kKS; ++mt) {
          acc[mt][0] *= al0; acc[mt][1] *= al1; acc[mt][2] *= al0; acc[mt][3] *= al1;
        }
      }
      auto weights = [&](const float (&x)[4], uint32_t& b0, uint32_t& b1) {
        const float2 shift = make_float2(kPShift, kPShift);
        const float2 lo = __ffma2_rn(__fadd2_rn(make_float2(x[0], x[1]), off), sc, shift);
        const float2 hi = __ffma2_rn(__fadd2_rn(make_float2(x[2], x[3]), off), sc, shift);
        const float e0 = fast_exp2(lo.x), e1 = fast_exp2(lo.y);
        const float e2 = fast_exp2(hi.x), e3 = fast_exp2(hi.y);
        l = __fadd2_rn(l, __fadd2_rn(make_float2(e0, e1), make_float2(e2, e3)));
        b0 = movmatrix_trans(pack_f16x2(e0, e1));
        b1 = movmatrix_trans(pack_f16x2(e2, e3));
      };
      uint32_t ps0, ps1, pu0, pu1;
      weights(s, ps0, ps1);
      weights(u, pu0, pu1);
      add_values<HD>(stage, places, ps0, ps1, acc);
      add_values<HD>(other, places, pu0, pu1, acc);
      stage = other + R::kStageBytes;
      if (stage == ring_end) stage = ring_at;
      __syncwarp();  // every lane is done with both
      copy();
      if (both) copy();
    }

    float l0 = l.x, l1 = l.y;
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, o);
      l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    }
    const float v_unit = g4.v_scale * kScaleUnit;
    if (seg == pages) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int col = k == 0 ? c0 : c1;
        if (col >= cols) continue;
        const float inv = v_unit / (k == 0 ? l0 : l1);
        const int j = col / a.group, hh = col - j * a.group;
        uint4* o = reinterpret_cast<uint4*>(
            a.out + (static_cast<size_t>(t0 + j) * a.nh + h * a.group + hh) * HD + g * kPer);
#pragma unroll
        for (int v = 0; v < kPer / 8; ++v) {
          auto two = [&](int mt) { return pack_bf16x2(acc[mt][k] * inv, acc[mt][k + 2] * inv); };
          o[v] = make_uint4(two(4 * v), two(4 * v + 1), two(4 * v + 2), two(4 * v + 3));
        }
      }
    } else {
      const size_t piece = static_cast<size_t>(first == 0 ? 2 * w + 1 : 2 * w);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int col = k == 0 ? c0 : c1;
        if (col >= cols) continue;
        float4* o = reinterpret_cast<float4*>(a.part_o + (piece * kMaxCols + col) * HD + g * kPer);
#pragma unroll
        for (int v = 0; v < kPer / 4; ++v)
          o[v] = make_float4(acc[2 * v][k], acc[2 * v][k + 2], acc[2 * v + 1][k],
                             acc[2 * v + 1][k + 2]);
        if (g == 0)
          a.part_ml[piece * kMaxCols + col] =
              k == 0 ? make_float2(l0 == 0.f ? -INFINITY : -off.x * sc0, l0)
                     : make_float2(l1 == 0.f ? -INFINITY : -off.y * sc1, l1);
      }
      // the last piece of this (request, kv head) to finish merges all of them
      const long long begin = static_cast<long long>(a.dec_off[r]) * a.nkv +
                              static_cast<long long>(h) * pages;
      const int w0 = stream.warp_of(begin), pieces = stream.warp_of(begin + pages - 1) - w0 + 1;
      __threadfence();
      __syncwarp();
      int prev = 0;
      if (lane == 0) prev = atomicAdd(a.done + r * a.nkv + h, 1);
      prev = __shfl_sync(0xffffffffu, prev, 0);
      if (prev == pieces - 1) {
        __threadfence();
        if (cols <= 4) merge_pieces<HD, 8>(a, w0, pieces, h, t0, cols, v_unit);
        else merge_pieces<HD, 4>(a, w0, pieces, h, t0, cols, v_unit);
      }
    }
  }
  copies_wait<0>();
  __syncwarp();
  if (bad) raise_error(a.err, RB_EBIT_BLOCK_ID);
}

}  // namespace attn
}  // namespace rb
