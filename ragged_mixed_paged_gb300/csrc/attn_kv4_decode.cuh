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
// A page of one kv head is 9 hd contiguous bytes of K and as many of V.  They go from memory to
// the registers of the lane whose MMA operand they are, without shared memory: the MMA does not
// mind which 16 values of head_dim (K) or which dims and keys (V) a step takes, as long as both operands
// agree, so the order is chosen to make a lane's bytes neighbours.  With g = lane / 4, t = lane % 4:
//   K  rows g and g + 8 of the MMA are keys kg = 4 (g / 2) + g % 2 and kg + 2; lane (g, t) holds
//      values [t hd / 4, (t + 1) hd / 4) of both, and step s takes its s-th four values;
//   V  row g of step s is dim (hd / 8) g + 2 s and row g + 8 the next one; the lane holds the hd / 8
//      values of dims [(hd / 8) g, ...) of keys 4t .. 4t + 3, whose codes are paired by two
//      shifts and masks for a word of eight: neighbouring codes then belong to neighbouring keys.
// A lane so ends up with hd / 8 neighbouring values of two columns of the output.
//
// Two pages a step, the next two steps' bytes on their way in registers (kDepth).
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

// One lane's bytes of a page of one kv head.
template <int HD>
struct Page {
  static constexpr int kWords = HD / 32;  // words of eight codes per K row; V words per key: half
  uint32_t k[2][kWords];
  uint32_t v[4][kWords / 2];
  uint32_t ks[2], vs;
};

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&r)[N], const uint8_t* p) {
  if constexpr (N == 4) {
    const uint4 w = __ldg(reinterpret_cast<const uint4*>(p));
    r[0] = w.x; r[1] = w.y; r[2] = w.z; r[3] = w.w;
  } else if constexpr (N == 2) {
    const uint2 w = __ldg(reinterpret_cast<const uint2*>(p));
    r[0] = w.x; r[1] = w.y;
  } else {
    r[0] = __ldg(reinterpret_cast<const uint32_t*>(p));
  }
}

// `k` and `v`: this lane's first bytes (codes of its first K row; codes of its first V key).
template <int HD>
__device__ __forceinline__ void load_page(Page<HD>& p, const uint8_t* k, const uint8_t* v,
                                          int k_scale_at, int v_scale_at) {
  load_words(p.k[0], k);
  load_words(p.k[1], k + 2 * (HD / 2));
#pragma unroll
  for (int i = 0; i < 4; ++i) load_words(p.v[i], v + i * (HD / 2));
  if constexpr (HD == 128) {
    p.ks[0] = __ldg(reinterpret_cast<const uint16_t*>(k + k_scale_at));
    p.ks[1] = __ldg(reinterpret_cast<const uint16_t*>(k + k_scale_at + 2 * (HD / 16)));
  } else {
    p.ks[0] = __ldg(k + k_scale_at);
    p.ks[1] = __ldg(k + k_scale_at + 2 * (HD / 16));
  }
  p.vs = __ldg(reinterpret_cast<const uint32_t*>(v + v_scale_at));
}

// S^T of a page: two chains of MMAs.
template <int HD>
__device__ __forceinline__ void scores(const Page<HD>& p, const uint32_t (&bq)[HD / 16][2],
                                       float (&s)[4]) {
  float s2[4] = {0.f, 0.f, 0.f, 0.f};
  s[0] = s[1] = s[2] = s[3] = 0.f;
  const uint32_t sc0 = scales2(p.ks[0]), sc1 = scales2(p.ks[1]);
#pragma unroll
  for (int w = 0; w < HD / 32; ++w) {
    // (a lane's HD / 4 values are one block of 16 for HD 64, two for 128)
    const uint32_t m0 = w < 2 ? low2(sc0) : high2(sc0), m1 = w < 2 ? low2(sc1) : high2(sc1);
    uint32_t x[4], y[4];
    kv4::values8(p.k[0][w], x);
    kv4::values8(p.k[1][w], y);
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

// O^T += V^T P^T of a page.
template <int HD>
__device__ __forceinline__ void add_values(const Page<HD>& p, uint32_t pb0, uint32_t pb1,
                                           float (&acc)[HD / 16][4]) {
  const uint32_t s01 = scales2(p.vs), s23 = scales2(p.vs >> 16);
#pragma unroll
  for (int w = 0; w < HD / 64; ++w) {
    // even and odd dims of a word, the first key of a pair in the low half of each byte
    auto even = [](uint32_t x, uint32_t y) { return (x & 0x0f0f0f0fu) | ((y << 4) & 0xf0f0f0f0u); };
    auto odd = [](uint32_t x, uint32_t y) { return ((x >> 4) & 0x0f0f0f0fu) | (y & 0xf0f0f0f0u); };
    uint32_t e01[4], o01[4], e23[4], o23[4];
    kv4::values8(even(p.v[0][w], p.v[1][w]), e01);
    kv4::values8(odd(p.v[0][w], p.v[1][w]), o01);
    kv4::values8(even(p.v[2][w], p.v[3][w]), e23);
    kv4::values8(odd(p.v[2][w], p.v[3][w]), o23);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      mma_f16(acc[4 * w + i], hmul2(e01[i], s01), hmul2(o01[i], s01), hmul2(e23[i], s23),
              hmul2(o23[i], s23), pb0, pb1);
  }
}

}  // namespace kv4d

// One decode warp: pulls (request, kv head, split) units from the shared counter until none
// are left; `first_unit` >= 0: its first unit, handed out statically.
template <int HD>
__device__ void decode_warp_kv4(const Kv4Args& g4, int first_unit) {
  using namespace kv4d;
  const AttnArgs& a = g4.a;
  constexpr int kKS = HD / 16, kPer = HD / 8;  // MMA steps; output values of a lane and column
  constexpr int kPages = 2;                    // pages a step
  constexpr int kDepth = 2;                    // steps in registers
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int n_units = a.header[kHNumDecodeUnits];
  const int sp = a.header[kHSplitPages];
  const int key_g = 4 * (g >> 1) + (g & 1);  // key of the lane's first K row
  // byte offsets of the lane in a page: K codes and scales, V codes and scales
  const int k_at = key_g * (HD / 2) + t * (HD / 8);
  const int k_scale_at = 8 * HD + key_g * (HD / 16) + t * (HD / 64) - k_at;
  const int v_at = 4 * t * (HD / 2) + g * (HD / 16);
  const int v_scale_at = 8 * HD + (g * (HD / 8) / 16) * 16 + 4 * t - v_at;
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
    Page<HD> buf[kDepth][kPages] = {};  // (a step's missing second page: any finite values)
    auto load = [&](Page<HD>& dst, int i) {  // pages in order; past the last one nothing
      if (i >= n_pages) return;
      if (i - win >= 32) {
        win += 32;
        bid = bid_next;
        bid_next = page(win + 32 + lane);
      }
      const int id = __shfl_sync(0xffffffffu, bid, i - win);
      const size_t at = (static_cast<size_t>(id) * a.nkv + h) * kv4::page_bytes(HD);
      load_page<HD>(dst, g4.k + at + k_at, g4.v + at + v_at, k_scale_at, v_scale_at);
    };
#pragma unroll
    for (int d = 0; d < kDepth; ++d)
#pragma unroll
      for (int p = 0; p < kPages; ++p) load(buf[d][p], d * kPages + p);

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

    auto step = [&](Page<HD> (&pg)[kPages], int i0) {
      float x[kPages][4];
      float g0 = -INFINITY, g1 = -INFINITY;
#pragma unroll
      for (int p = 0; p < kPages; ++p) {
        scores<HD>(pg[p], bq, x[p]);
        // keys past the end of the unit's pages (an odd last step) and of the column
        const int key = i0 + p < n_pages ? (p_begin + i0 + p) * kPage + key_g : 0x7ffffff0;
        x[p][0] = key <= lim0 ? x[p][0] * sc0 : -INFINITY;
        x[p][1] = key <= lim1 ? x[p][1] * sc1 : -INFINITY;
        x[p][2] = key + 2 <= lim0 ? x[p][2] * sc0 : -INFINITY;
        x[p][3] = key + 2 <= lim1 ? x[p][3] * sc1 : -INFINITY;
        g0 = fmax3(g0, x[p][0], x[p][2]);
        g1 = fmax3(g1, x[p][1], x[p][3]);
      }
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
#pragma unroll
      for (int p = 0; p < kPages; ++p) {
        const float e0 = fast_exp2(x[p][0] - ms0), e1 = fast_exp2(x[p][1] - ms1);
        const float e2 = fast_exp2(x[p][2] - ms0), e3 = fast_exp2(x[p][3] - ms1);
        l0 += e0 + e2;
        l1 += e1 + e3;
        add_values<HD>(pg[p], movmatrix_trans(pack_f16x2(e0, e1)),
                       movmatrix_trans(pack_f16x2(e2, e3)), acc);
      }
    };
    for (int i = 0; i < n_pages; i += kDepth * kPages) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) {
        const int i0 = i + d * kPages;
        if (i0 >= n_pages) break;
        step(buf[d], i0);
#pragma unroll
        for (int p = 0; p < kPages; ++p) load(buf[d][p], i0 + kDepth * kPages + p);
      }
    }
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
