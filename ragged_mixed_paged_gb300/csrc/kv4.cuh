// The 4-bit cache's format: where a token's codes and scales are, and the conversions.  Not part of
// the C ABI (rb.h states the format).
//
// A page of one kv head is 9 hd contiguous bytes: 16 tokens x hd / 2 bytes of codes, then hd scale
// bytes, [16 tokens][hd / 16] for keys and [hd / 16][16 tokens] for values.  Keys and values
// are read by different operands of the attention's MMAs: a lane needs the scales of few keys
// and neighbouring blocks of K, of one block and neighbouring keys of V.  The bytes that one
// token owns are its own (never half of a byte that another token writes).
#pragma once

#include <cuda_fp16.h>

#include "rb_internal.cuh"

namespace rb {
namespace kv4 {

constexpr int kPage = 16;   // tokens per page
constexpr int kBlock = 16;  // values that share a scale

__host__ __device__ constexpr int page_bytes(int hd) { return 9 * hd; }  // of one kv head

// A layer's scale.  The range keeps it, its reciprocal and their products with what the kernels fold
// into them (2^8, log2 e) ordinary fp32 numbers.
inline bool layer_scale_ok(float s) { return s >= 0x1p-100f && s <= 0x1p100f; }

// Byte offset of the codes of (slot, head, block of 16 values), 8 bytes, and of their scale.
struct Place {
  size_t code, scale;
};
template <bool kValues>
__device__ __forceinline__ Place place(int slot, int head, int block, int nkv, int hd) {
  const int tok = slot & (kPage - 1);
  const size_t base = (static_cast<size_t>(slot >> 4) * nkv + head) * page_bytes(hd);
  return {base + tok * (hd / 2) + block * 8,
          base + 8 * hd + (kValues ? block * kPage + tok : tok * (hd / kBlock) + block)};
}

// Scale byte of max / 6 (round to nearest even, 448 at most) and its value.
__device__ __forceinline__ uint32_t scale_byte(float six) {
  uint16_t b;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(b) : "f"(0.f), "f"(six));
  return b & 0x7fu;
}
// Exact: four bits of exponent and three of mantissa, moved into a half's fields, are the value
// times 2^-8 (the biases are 7 and 15); 0x7f, which is not written, is 480, and bit 7 is ignored,
// so that a scale is finite whatever a page holds.
__device__ __forceinline__ float scale_value(uint32_t b) {
  return __half2float(__ushort_as_half(static_cast<unsigned short>((b & 0x7fu) << 7))) * 256.f;
}

// Four codes (two bytes) from four values: nearest, ties to the even code, 6 at most.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  uint16_t r;
  asm("{\n\t.reg .b8 x, y;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 x, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 y, %4, %3;\n\t"
      "mov.b16 %0, {x, y};\n\t}"
      : "=h"(r)
      : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}

// a / b, correctly rounded for ordinary values: a product with the rounded reciprocal and one
// correction by its exact remainder (Markstein 1990), three instructions once r = 1 / b is there.
// The remainder is q b - a, so that the quotient of -0 is -0.
__device__ __forceinline__ float quotient(float a, float b, float r) {
  const float q = a * r;
  return fmaf(-fmaf(q, b, -a), r, q);
}
__device__ __forceinline__ float2 quotient(float2 a, float b, float r) {
  const float2 r2 = make_float2(r, r), q = __fmul2_rn(a, r2);
  const float2 rest = __ffma2_rn(q, make_float2(b, b), make_float2(-a.x, -a.y));
  return __ffma2_rn(rest, make_float2(-r, -r), q);
}

// The eight values of four bytes of codes as half2 (value 2i in the low half), exact.
__device__ __forceinline__ void values8(uint32_t codes, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\tcvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\tcvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(codes));
}

}  // namespace kv4
}  // namespace rb
