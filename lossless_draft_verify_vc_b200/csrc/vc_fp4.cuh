// vc_fp4.cuh -- the 4-bit floating-point draft cache's number format and
// record layout (include/vc.h, "4-bit floating-point draft cache"): e2m1
// codes, one e4m3 scale per 16 channels of a token, 16 tokens per record.
#pragma once

#include "vc_common.cuh"

namespace vc {
namespace fp4 {

constexpr int kTok = 16;  // tokens per record

template <int D>
struct Rec {
  static constexpr int BYTES = 18 * D;
  static constexpr int V = 8 * D;    // value codes
  static constexpr int KS = 16 * D;  // key scales
  static constexpr int VS = 17 * D;  // value scales
};

// 8 e2m1 codes of a word -> 4 x f16x2 (channel pairs, exact).  Pass whole
// words: with a byte zero-extended to a word and three of the results unused,
// CUDA 12.9 compiled the conversion to zeros.
__device__ __forceinline__ void codes_to_h2(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}\n"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}

// Two e4m3 scales (bits 0..15) -> f16x2 (exact).
__device__ __forceinline__ uint32_t scales_to_h2(uint32_t w) {
  uint32_t o;
  asm("{\n\t.reg .b16 a;\n\t"
      "cvt.u16.u32 a, %1;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t}\n"
      : "=r"(o)
      : "r"(w));
  return o;
}

__device__ __forceinline__ float scale_to_float(uint8_t s) { return unpack_h2(scales_to_h2(s)).x; }

// e4m3 of x >= 0, to nearest even, saturating at 448.
__device__ __forceinline__ uint8_t float_to_scale(float x) {
  uint32_t o;
  asm("{\n\t.reg .b16 a;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 a, 0f00000000, %1;\n\t"
      "cvt.u32.u16 %0, a;\n\t}\n"
      : "=r"(o)
      : "f"(x));
  return static_cast<uint8_t>(o);
}

// 8 floats -> 8 e2m1 codes (element i in bits 4i), to nearest even, saturating.
__device__ __forceinline__ uint32_t floats_to_codes(const float* x) {
  uint32_t o;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}\n"
      : "=r"(o)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return o;
}

// Quotients of numbers with few significant bits, as the roundings below need
// them: x * (hi + lo) with hi + lo = 1 / d up to 2^-42 of itself is off by so
// little that one fp32 rounding returns x / d itself where that is a number
// of at most 20 significant bits, such as the border between two codes (e2m1:
// 3 bits, e4m3: 5).  Any other x / d differs from a border by at least 2^-11
// of it (x has at most 11 bits -- bf16, fp16 -- and border * d at most 8), so
// every rounding decides as exact division does.  hi is below 1 / d, so that
// lo >= 0 and a zero keeps its sign (x = -0: -0 + -0; with lo < 0 it would be
// -0 + +0 = +0).
struct Recip {
  float hi, lo;
  __device__ __forceinline__ float2 times(float2 x) const {  // two numbers per instruction
    return __ffma2_rn(x, make_float2(hi, hi), __fmul2_rn(x, make_float2(lo, lo)));
  }
};
__device__ __forceinline__ Recip recip(float d) {  // 1 / d for d > 0
  Recip r;
  asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r.hi) : "f"(d));
  // (off by at most one step; two steps down it is 1 to 3 below)
  r.hi = __int_as_float(__float_as_int(r.hi) - 2);
  r.lo = fmaf(-d, r.hi, 1.f) * r.hi;
  return r;
}

constexpr float kMaxAbs = 6.f * 448.f;  // largest value in the scales' range

// The scale of a block whose largest |x| * 2^-exp is amax <= kMaxAbs.
__device__ __forceinline__ uint8_t block_scale(float amax) {
  constexpr float hi = 1.f / 6.f, lo = static_cast<float>(1.0 / 6.0 - static_cast<double>(hi));
  return float_to_scale(fmaf(amax, hi, amax * lo));
}

// Codes of N values x of one block under the scale s8; down: the head's 2^-exp.
template <int N>
__device__ __forceinline__ void quantise_codes(float (&x)[N], uint8_t s8, float down, uint32_t (&codes)[N / 8]) {
  const float s = scale_to_float(s8);
  Recip r = recip(s);  // (s = 0: not used)
  r.hi *= down, r.lo *= down;
#pragma unroll
  for (int i = 0; i < N; i += 2) {
    const float2 y = r.times(make_float2(x[i], x[i + 1]));
    x[i] = y.x, x[i + 1] = y.y;
  }
#pragma unroll
  for (int i = 0; i < N / 8; ++i) codes[i] = s > 0.f ? floats_to_codes(x + 8 * i) : 0u;
}

}  // namespace fp4
}  // namespace vc
