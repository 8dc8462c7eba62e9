// vc_fp4.cuh -- the 4-bit floating-point draft cache's number format and
// record layout (include/vc.h, "4-bit floating-point draft cache"): e2m1
// codes, one e4m3 scale per 16 channels of a token, 16 tokens per record.
#pragma once

#include "vc_common.cuh"

namespace vc {
namespace fp4 {

constexpr int kTok = 16;  // tokens per record
constexpr int kBlk = 16;  // channels per scale

template <int D>
struct Rec {
  static constexpr int BYTES = 18 * D;
  static constexpr int V = 8 * D;    // value codes
  static constexpr int KS = 16 * D;  // key scales
  static constexpr int VS = 17 * D;  // value scales
  static constexpr int BLKS = D / kBlk;
  // Offsets for token t of the record and 16-channel block j; a block's key
  // codes are 8 contiguous bytes, its value codes two 4-byte words of 8
  // channels each (contiguous when D == 128).
  __host__ __device__ static constexpr int k_codes(int t, int j) { return t * (D / 2) + j * 8; }
  __host__ __device__ static constexpr int v_word(int t, int j, int half) {
    return D == 128 ? V + (t >> 3) * 512 + j * 64 + ((t & 7) >> 1) * 16 + (t & 1) * 8 + half * 4
                    : V + (2 * j + half) * 64 + ((t & 7) >> 1) * 16 + (t >> 3) * 8 + (t & 1) * 4;
  }
  __host__ __device__ static constexpr int k_scale(int t, int j) {
    return D == 128 ? KS + (t & 7) * 16 + (j >> 1) * 4 + (t >> 3) * 2 + (j & 1) : KS + (t & 7) * 8 + j * 2 + (t >> 3);
  }
  __host__ __device__ static constexpr int v_scale(int t, int j) {
    return VS + j * 16 + ((t & 7) >> 1) * 4 + (t >> 3) * 2 + (t & 1);
  }
};

// A head's power of two (clamped so that it and its inverse are normal).
__device__ __forceinline__ float two_to(const int32_t* exp, int h, int sign) {
  if (!exp) return 1.f;
  const int e = min(60, max(-60, __ldg(exp + h))) * sign;
  return __int_as_float((e + 127) << 23);
}

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

// One block of 16 values (already multiplied by 2^-exp) -> codes and scale.
// x / s is taken as x * (1 / s), off by at most 2^-22 of itself, and rounded
// to 17 significant bits before the e2m1 rounding.  That decides as exact
// division does: a border m between two codes has <= 3 significant bits, s
// has 4 and x at most 11 (bf16, fp16), so x / s either is m, and the rounding
// to 17 bits returns m itself, or differs from it by at least 2^-11 of m,
// which an error of 2^-17 does not bridge.  The scale's own x / 6 is one IEEE
// division (its borders have 5 bits, so the same argument holds).
// Returns true when a value was NaN or outside the scales' range.
__device__ __forceinline__ bool quantise_block(float (&x)[16], uint32_t (&codes)[2], uint8_t& s8) {
  bool odd = false;
  float amax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const bool nan = x[i] != x[i];
    odd |= nan;
    x[i] = nan ? 0.f : x[i];
    amax = fmaxf(amax, fabsf(x[i]));
  }
  odd |= amax > 2688.f;
  s8 = float_to_scale(__fdiv_rn(amax, 6.f));
  const float s = scale_to_float(s8);
  if (s == 0.f) {
    codes[0] = codes[1] = 0u;
    return odd;
  }
  const float r = __frcp_rn(s);
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = __int_as_float((__float_as_int(x[i] * r) + 0x40) & ~0x7f);
  codes[0] = floats_to_codes(x);
  codes[1] = floats_to_codes(x + 8);
  return odd;
}

}  // namespace fp4
}  // namespace vc
