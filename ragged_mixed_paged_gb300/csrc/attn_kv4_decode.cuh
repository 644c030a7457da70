// Split-KV decode warp of the attention over a 4-bit cache.  Not part of the C ABI.
//
// Work unit = (request, kv head, split of pages), one warp per unit, as in the 16-bit cache's
// decode; the contraction runs transposed, a 16-token page per MMA tile:
//   S^T[16 keys, 8 cols] = K[16, hd] . Q^T[hd, 8]     cols = (query token, head of the group)
//   O^T[hd, 8 cols]     += V^T[hd, 16] . P^T[16, 8]
// with mma.sync m16n8k16, fp16 in and fp32 accumulated.  Every value that the cache can hold is
// exact in fp16 (two bits of a code times four of a scale, between 2^-10 and 2880), so K and V enter
// the MMAs unrounded; Q is divided by a power of two per column, which keeps its 8 bits.
//
// A page of one kv head is 9 hd contiguous bytes of K and as many of V.  A warp copies them to its
// own ring in shared memory with 16-byte cp.async, kStages pages ahead, and each lane then reads the
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
// What bounds it: the codes' conversions.  A page costs 64 of them per lane (hd 128), two cycles
// each on the pipe that also takes masks, shifts and comparisons, about 285 cycles a page of
// 2304 bytes in all, where HBM delivers one to a quarter SM in 390.
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

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&a),
                            *reinterpret_cast<const __half2*>(&b));
  return *reinterpret_cast<const uint32_t*>(&v);
}
// Scale bytes 0 and 1 of `w` as a half2 (kv4::scale_value of each).
__device__ __forceinline__ uint32_t scales2(uint32_t w) {
  return hmul2((w & 0x7fu) << 7 | (w & 0x7f00u) << 15, 0x5c005c00u);  // times 256
}
__device__ __forceinline__ uint32_t low2(uint32_t w) { return __byte_perm(w, w, 0x1010); }
__device__ __forceinline__ uint32_t high2(uint32_t w) { return __byte_perm(w, w, 0x3232); }

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7},"
      " {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Geometry of a warp's ring: pages as they lie in the cache, but for the order of rows (and, in
// rows of 64 bytes, of 16-byte chunks), which keeps the lanes' reads free of bank conflicts.
//   K: the lanes' first rows, in order of g, then their second ones: lane's bytes at lane x hd / 8
//   V: row 4t + i at t + 4i; chunk c of it at c ^ 2 for t >= 2 (hd 128)
template <int HD>
struct Ring {
  static constexpr int kStages = 4;              // pages
  static constexpr int kBytes = 9 * HD;          // K or V of a page
  static constexpr int kStageBytes = 2 * kBytes;
  static constexpr int kWarpBytes = kStages * kStageBytes;
  static constexpr int kRow = HD / 2;            // bytes of codes of a row
  static constexpr int kCopies = (kBytes / 16 + 31) / 32;
};

__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {  // all but the last N groups have landed
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Where chunk i of a page of K (V) goes in its stage.
template <int HD, bool kValues>
__device__ __forceinline__ int chunk_at(int i) {
  constexpr int kPerRow = HD / 32;  // chunks of codes of a row
  if (i >= 8 * HD / 16) return i * 16;  // scales stay where they are
  const int r = i / kPerRow, c = i % kPerRow;
  if (kValues) return ((r >> 2) + 4 * (r & 3)) * (HD / 2) + ((HD == 128 ? c ^ ((r >> 3) * 2) : c) << 4);
  return (((r >> 2) * 2 + (r & 1)) + 8 * ((r >> 1) & 1)) * (HD / 2) + (c << 4);
}

template <int N>
__device__ __forceinline__ void read_words(uint32_t (&r)[N], const uint8_t* p) {
  if constexpr (N == 4) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    r[0] = w.x; r[1] = w.y; r[2] = w.z; r[3] = w.w;
  } else if constexpr (N == 2) {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    r[0] = w.x; r[1] = w.y;
  } else {
    r[0] = *reinterpret_cast<const uint32_t*>(p);
  }
}

// S^T of the page whose K is at `k`: two chains of MMAs.
template <int HD>
__device__ __forceinline__ void scores(const uint8_t* k, int lane, const uint32_t (&bq)[HD / 16][2],
                                       float (&s)[4]) {
  const int g = lane >> 2, t = lane & 3, key_g = 4 * (g >> 1) + (g & 1);
  float s2[4] = {0.f, 0.f, 0.f, 0.f};
  s[0] = s[1] = s[2] = s[3] = 0.f;
  uint32_t c0[HD / 32], c1[HD / 32];
  read_words(c0, k + lane * (HD / 8));
  read_words(c1, k + 4 * HD + lane * (HD / 8));
  const uint8_t* sp = k + 8 * HD + key_g * (HD / 16) + t * (HD / 64);
  uint32_t sc0, sc1;
  if constexpr (HD == 128) {
    sc0 = scales2(*reinterpret_cast<const uint16_t*>(sp));
    sc1 = scales2(*reinterpret_cast<const uint16_t*>(sp + 2 * (HD / 16)));
  } else {
    sc0 = scales2(*sp);
    sc1 = scales2(*(sp + 2 * (HD / 16)));
  }
#pragma unroll
  for (int w = 0; w < HD / 32; ++w) {
    // (a lane's HD / 4 values are one block of 16 for HD 64, two for 128)
    const uint32_t m0 = w < 2 ? low2(sc0) : high2(sc0), m1 = w < 2 ? low2(sc1) : high2(sc1);
    uint32_t x[4], y[4];
    kv4::values8(c0[w], x);
    kv4::values8(c1[w], y);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = hmul2(x[i], m0);
      y[i] = hmul2(y[i], m1);
    }
    mma_f16(s, x[0], y[0], x[1], y[1], bq[2 * w][0], bq[2 * w][1]);
    mma_f16(s2, x[2], y[2], x[3], y[3], bq[2 * w + 1][0], bq[2 * w + 1][1]);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) s[i] += s2[i];
}

// O^T += V^T P^T of the page whose V is at `v`.
template <int HD>
__device__ __forceinline__ void add_values(const uint8_t* v, int lane, uint32_t pb0, uint32_t pb1,
                                           float (&acc)[HD / 16][4]) {
  const int g = lane >> 2, t = lane & 3;
  const uint32_t sv = *reinterpret_cast<const uint32_t*>(
      v + 8 * HD + (g * (HD / 8) / 16) * 16 + 4 * t);
  const uint32_t s01 = scales2(sv), s23 = scales2(sv >> 16);
  uint32_t c[4][HD / 64];
  const int chunk = g * (HD / 16) / 16, in = g * (HD / 16) % 16;
  const uint8_t* p = v + t * (HD / 2) + ((HD == 128 ? chunk ^ ((t >> 1) * 2) : chunk) << 4) + in;
#pragma unroll
  for (int i = 0; i < 4; ++i) read_words(c[i], p + 4 * i * (HD / 2));
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
    for (int i = 0; i < 4; ++i)
      mma_f16(acc[4 * w + i], hmul2(e01[i], s01), hmul2(o01[i], s01), hmul2(e23[i], s23),
              hmul2(o23[i], s23), pb0, pb1);
  }
}

}  // namespace kv4d

// One decode warp: pulls (request, kv head, split) units from the shared counter until none
// are left; `ring` is its kv4d::Ring in shared memory, `first_unit` >= 0 its first unit, handed out
// statically.
template <int HD>
__device__ void decode_warp_kv4(const Kv4Args& g4, uint8_t* ring, int first_unit) {
  using namespace kv4d;
  const AttnArgs& a = g4.a;
  constexpr int kKS = HD / 16, kPer = HD / 8;  // MMA steps; output values of a lane and column
  using R = Ring<HD>;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n_units = a.header[kHNumDecodeUnits];
  const int sp = a.header[kHSplitPages];
  const int key_g = 4 * (g >> 1) + (g & 1);  // key of the lane's first K row
  const uint32_t ring_at = smem_u32(ring);
  int k_to[R::kCopies], v_to[R::kCopies];  // where this lane's chunks go in a stage
#pragma unroll
  for (int i = 0; i < R::kCopies; ++i) {
    k_to[i] = chunk_at<HD, false>(lane + 32 * i);
    v_to[i] = R::kBytes + chunk_at<HD, true>(lane + 32 * i);
  }
  int next_static = first_unit;
  while (true) {
    int u = next_static;
    if (u < 0) {
      if (lane == 0) u = atomicAdd(a.header + kHDecodeNext, 1);
      u = __shfl_sync(0xffffffffu, u, 0);
    }
    next_static = -1;
    if (u >= n_units) break;
    const int r = warp_upper_bound_i32(a.dec_off, a.R + 1, u) - 1;
    const int first = a.dec_off[r];
    const int nsplit = (a.dec_off[r + 1] - first) / a.nkv;
    const int local = u - first;
    const int split = local / a.nkv, h = local - split * a.nkv;
    const int t0 = a.qsl[r], q = a.qsl[r + 1] - t0, L = a.seq_lens[r];
    const int c = L - q, cols = q * a.group, pages = (L + kPage - 1) / kPage;
    const int p_begin = split * sp, n_pages = min(p_begin + sp, pages) - p_begin;

    // page ids of pages [win, win + 32) held one per lane, the next window prefetched
    const int32_t* bt_row = a.block_table + static_cast<size_t>(r) * a.MB;
    int win = 0;
    bool bad = false;
    auto page = [&](int i) {
      if (i >= n_pages) return a.null_block;
      const int id = kernel_page(bt_row, p_begin + i, a.ratio, a.num_blocks, a.null_block);
      bad |= id < 0;
      return id < 0 ? a.null_block : id;
    };
    int bid = page(lane), bid_next = page(32 + lane);
    auto load = [&](int i) {  // pages in order; past the last one an empty group
      if (i < n_pages) {
        if (i - win >= 32) {
          win += 32;
          bid = bid_next;
          bid_next = page(win + 32 + lane);
        }
        const int id = __shfl_sync(0xffffffffu, bid, i - win);
        const size_t at = (static_cast<size_t>(id) * a.nkv + h) * kv4::page_bytes(HD) + lane * 16;
        const uint32_t to = ring_at + (i % R::kStages) * R::kStageBytes;
#pragma unroll
        for (int c = 0; c < R::kCopies; ++c) {
          if ((c + 1) * 32 <= R::kBytes / 16 || lane < R::kBytes / 16 - c * 32) {
            copy16(to + k_to[c], g4.k + at + c * 512);
            copy16(to + v_to[c], g4.v + at + c * 512);
          }
        }
      }
      copies_commit();
    };
#pragma unroll
    for (int i = 0; i < R::kStages - 1; ++i) load(i);

    // Q^T fragments: column g, values [t hd / 4, (t + 1) hd / 4) over 2^e
    uint32_t bq[kKS][2];
    float up;
    {
      const bool valid = g < cols;
      const int j = valid ? g / a.group : 0;
      const int hh = valid ? g - j * a.group : 0;
      const uint4* qp = reinterpret_cast<const uint4*>(
          a.q + (static_cast<size_t>(t0 + j) * a.nh + h * a.group + hh) * HD + t * (HD / 4));
      uint4 w[HD / 32];
#pragma unroll
      for (int i = 0; i < HD / 32; ++i) w[i] = valid ? __ldg(qp + i) : make_uint4(0u, 0u, 0u, 0u);
      float f[HD / 4], top = 0.f;
#pragma unroll
      for (int i = 0; i < HD / 8; ++i) {
        const uint32_t x = reinterpret_cast<const uint32_t*>(w)[i];
        f[2 * i] = __uint_as_float(x << 16);
        f[2 * i + 1] = __uint_as_float(x & 0xffff0000u);
        top = fmax3(top, fabsf(f[2 * i]), fabsf(f[2 * i + 1]));
      }
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      float down;
      power_of(top, &down, &up);
#pragma unroll
      for (int s = 0; s < kKS; ++s)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          bq[s][i] = pack_f16x2(f[4 * s + 2 * i] * down, f[4 * s + 2 * i + 1] * down);
    }
    // the lane's columns of S^T: their scales and their last visible key
    const int c0 = 2 * t, c1 = c0 + 1;
    const float sc0 = __shfl_sync(0xffffffffu, up, 4 * c0) * a.scale_log2;
    const float sc1 = __shfl_sync(0xffffffffu, up, 4 * c1) * a.scale_log2;
    const int lim0 = c0 < cols ? c + c0 / a.group : c;
    const int lim1 = c1 < cols ? c + c1 / a.group : c;
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float acc[kKS][4];
#pragma unroll
    for (int mt = 0; mt < kKS; ++mt) acc[mt][0] = acc[mt][1] = acc[mt][2] = acc[mt][3] = 0.f;

    for (int i = 0; i < n_pages; ++i) {
      copies_wait<R::kStages - 2>();
      __syncwarp();  // page i has landed for every lane, and every lane is done with page i - 1
      load(i + R::kStages - 1);
      const uint8_t* stage = ring + (i % R::kStages) * R::kStageBytes;
      float x[4];
      scores<HD>(stage, lane, bq, x);
      const int key = (p_begin + i) * kPage + key_g;
      x[0] *= sc0;
      x[1] *= sc1;
      x[2] *= sc0;
      x[3] *= sc1;
      if ((p_begin + i) * kPage + kPage - 1 > c) {  // (the columns' last keys are c and more)
        x[0] = key <= lim0 ? x[0] : -INFINITY;
        x[1] = key <= lim1 ? x[1] : -INFINITY;
        x[2] = key + 2 <= lim0 ? x[2] : -INFINITY;
        x[3] = key + 2 <= lim1 ? x[3] : -INFINITY;
      }
      float g0 = fmaxf(x[0], x[2]), g1 = fmaxf(x[1], x[3]);
      // exponents against a reference that moves only when a score exceeds it by more than
      // kGrowth (log2 units), so that P stays below 2^(kPShift + kGrowth)
      constexpr float kGrowth = 8.f;
      if (__any_sync(0xffffffffu, g0 > m0 + kGrowth || g1 > m1 + kGrowth)) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
          g0 = fmaxf(g0, __shfl_xor_sync(0xffffffffu, g0, o));
          g1 = fmaxf(g1, __shfl_xor_sync(0xffffffffu, g1, o));
        }
        const float mn0 = fmaxf(m0, g0), mn1 = fmaxf(m1, g1);
        const float al0 = fast_exp2(m0 - (mn0 == -INFINITY ? 0.f : mn0));
        const float al1 = fast_exp2(m1 - (mn1 == -INFINITY ? 0.f : mn1));
        l0 *= al0;
        l1 *= al1;
#pragma unroll
        for (int mt = 0; mt < kKS; ++mt) {
          acc[mt][0] *= al0; acc[mt][1] *= al1; acc[mt][2] *= al0; acc[mt][3] *= al1;
        }
        m0 = mn0;
        m1 = mn1;
      }
      const float ms0 = m0 == -INFINITY ? 0.f : m0 - kPShift;
      const float ms1 = m1 == -INFINITY ? 0.f : m1 - kPShift;
      const float e0 = fast_exp2(x[0] - ms0), e1 = fast_exp2(x[1] - ms1);
      const float e2 = fast_exp2(x[2] - ms0), e3 = fast_exp2(x[3] - ms1);
      l0 += e0 + e2;
      l1 += e1 + e3;
      add_values<HD>(stage + R::kBytes, lane, movmatrix_trans(pack_f16x2(e0, e1)),
                     movmatrix_trans(pack_f16x2(e2, e3)), acc);
    }
    copies_wait<0>();
    __syncwarp();  // every lane is done with the ring
    if (bad) raise_error(a.err, RB_EBIT_BLOCK_ID);

#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
      l0 += __shfl_xor_sync(0xffffffffu, l0, o);
      l1 += __shfl_xor_sync(0xffffffffu, l1, o);
    }
    if (nsplit == 1) {
      const float inv0 = l0 > 0.f ? g4.v_scale / l0 : 0.f, inv1 = l1 > 0.f ? g4.v_scale / l1 : 0.f;
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int col = k == 0 ? c0 : c1;
        if (col >= cols) continue;
        const float inv = k == 0 ? inv0 : inv1;
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
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float4* o = reinterpret_cast<float4*>(
            a.part_o + (static_cast<size_t>(u) * kMaxCols + (k == 0 ? c0 : c1)) * HD + g * kPer);
#pragma unroll
        for (int v = 0; v < kPer / 4; ++v)
          o[v] = make_float4(acc[2 * v][k] * g4.v_scale, acc[2 * v][k + 2] * g4.v_scale,
                             acc[2 * v + 1][k] * g4.v_scale, acc[2 * v + 1][k + 2] * g4.v_scale);
      }
      if (lane < 4) {
        a.part_ml[static_cast<size_t>(u) * kMaxCols + c0] = make_float2(m0, l0);
        a.part_ml[static_cast<size_t>(u) * kMaxCols + c1] = make_float2(m1, l1);
      }
      // the last split of this (request, kv head) to finish merges all partials
      __threadfence();
      __syncwarp();
      int prev = 0;
      if (lane == 0) prev = atomicAdd(a.done + r * a.nkv + h, 1);
      prev = __shfl_sync(0xffffffffu, prev, 0);
      if (prev == nsplit - 1) {
        __threadfence();
        combine_splits<HD, false>(a, h, first, nsplit, t0, cols);
      }
    }
  }
}

}  // namespace attn
}  // namespace rb
