// The 4-bit cache format on the device: encoding one lane's 8 channels and
// expanding codes to exact bf16 values.
//
// A head row of d values has 4 groups of d / 4.  A group's scale is a byte
// e << 3 | m of value 2^(e - 20) (1 + m / 8) (255 = NaN), a value is
// (code - 8) * scale.  code - 8 has at most 4 significant bits and the scale
// has 4, so every value is exact in bf16 (8 significant bits).
#pragma once

#include "msa_common.cuh"
#include "msa_sm100.cuh"

namespace msa {
namespace kv4 {

constexpr int kGroups = 4;            // scales of a head row
constexpr uint32_t kScaleNaN = 255u;  // a group that held a NaN or an infinity
constexpr uint32_t kScaleMax = 254u;

// bf16 bits of a scale: the byte is the top of a bf16 mantissa, its exponent moved by 127 - 20.
__device__ __forceinline__ uint32_t scale_bf16(uint32_t byte) {
  return byte == kScaleNaN ? 0x7FFFu : (byte << 4) + (107u << 7);
}
__device__ __forceinline__ float scale_f32(uint32_t byte) { return __uint_as_float((byte << 20) + (107u << 23)); }

__device__ __forceinline__ uint32_t hfma2_bf16(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("fma.rn.bf16x2 %0, %1, %2, %3;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
__device__ __forceinline__ uint32_t hmul2_bf16(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}
// -136 * scale of both halves: exact (136 = 17 * 8 and the scale's mantissa is at most 15, 17 * 15 = 255).
__device__ __forceinline__ uint32_t scale_bias(uint32_t s2) { return hmul2_bf16(s2, 0xC308C308u); }

// Nibble n (0..3) of both 16-bit halves of w as two bf16 values: 0x4300 | code is the bf16 128 + code, and
// (128 + code) s - 136 s is exact under one rounding because the result is.
__device__ __forceinline__ uint32_t and_or(uint32_t a, uint32_t b, uint32_t c) {  // (a & b) | c in one instruction
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
template <int N>
__device__ __forceinline__ uint32_t expand(uint32_t w, uint32_t s2, uint32_t b2) {
  return hfma2_bf16(and_or(w >> (4 * N), 0x000F000Fu, 0x43004300u), s2, b2);
}

// A word's 8 channels in order, as 4 bf16 pairs: nibble n of the low half is channel 2n, of the high half 2n + 1.
__device__ __forceinline__ uint4 expand8(uint32_t w, uint32_t s2, uint32_t b2) {
  return make_uint4(expand<0>(w, s2, b2), expand<1>(w, s2, b2), expand<2>(w, s2, b2), expand<3>(w, s2, b2));
}

// The same expansion for a kernel bound by its integer instructions.  The low byte of a half, masked to one of
// its nibbles, is already a bf16 proportional to the code: as bits of a subnormal (or of the first binade, where
// the spacing is the same) c << 0 is c 2^-133 and c << 4 is 16 c 2^-133.  So half the shifts and every OR go, and
//   c 2^-133 * M - 8 s 2^-18 = (c - 8) s 2^-18,  M = s 2^115 (or M / 16),
// is exact: all values come out scaled by 2^-18, which their user takes back in fp32.  M stays below 2^127.
constexpr float kSubUnscale = 262144.0f;                 // 2^18
constexpr uint32_t kSubScaleBias = (107u + 115u) << 7;   // M's bits are (byte << 4) + this
struct SubScale {
  uint32_t m, m16, b;
};
__device__ __forceinline__ SubScale sub_scale(uint32_t m) {
  SubScale s;
  s.m = m;
  s.m16 = hmul2_bf16(m, 0x3D803D80u);  // 2^-4
  s.b = hmul2_bf16(m, 0x80088008u);    // -8 * 2^-133
  return s;
}
__device__ __forceinline__ uint4 expand8_sub(uint32_t w, const SubScale& s) {
  const uint32_t h = w >> 8;
  return make_uint4(hfma2_bf16(w & 0x000F000Fu, s.m, s.b), hfma2_bf16(w & 0x00F000F0u, s.m16, s.b),
                    hfma2_bf16(h & 0x000F000Fu, s.m, s.b), hfma2_bf16(h & 0x00F000F0u, s.m16, s.b));
}

// The scale of a group whose largest magnitude is the bf16 `amax` (bits, finite): the smallest one with
// 7 scale >= amax.  The top mantissa bits of amax / 7 give it or the one below it, and 7 scale is exact.
__device__ __forceinline__ uint32_t scale_of(uint32_t amax_bits) {
  const float a = __uint_as_float(amax_bits << 16);
  int b = (int)(__float_as_uint(a * (1.0f / 7.0f)) >> 20) - (107 << 3);
  b = min(max(b, 0), (int)kScaleMax);
  if (7.0f * scale_f32((uint32_t)b) < a) ++b;
  return (uint32_t)min(b, (int)kScaleMax);
}

// The 8 codes of 4 channel pairs, round-to-nearest-even(x / s) + 8 for |x / s| <= 7: pair j's in nibble j of the halves.
// x has 8 and s has 4 significant bits, so x / s is a tie or at least 2^-11 away from one wherever it rounds to a
// code that is not 0.  fma(x, 1/s, 1.5 * 2^10) rounds x / s to a multiple of 2^-13 (1/s may be 2^-20 off): a tie is
// exact again, the others keep their side.  Adding 1.5 * 2^23 - 1.5 * 2^10 rounds that to an integer, which the
// mantissa then holds; its bits are summed with weights 16^i and the constant part taken off at the end.
__device__ __forceinline__ uint32_t codes8(const uint64_t (&x2)[4], float inv_s) {
  const uint64_t inv2 = f2_pack(inv_s, inv_s), half = f2_pack(1536.0f, 1536.0f);
  const uint64_t rest = f2_pack(12582912.0f - 1536.0f, 12582912.0f - 1536.0f);
  uint32_t lo = 0, hi = 0;
#pragma unroll
  for (int j = 3; j >= 0; --j) {
    float a, b;
    f2_unpack(f2_add(f2_fma(x2[j], inv2, half), rest), a, b);
    lo = lo * 16u + __float_as_uint(a);
    hi = hi * 16u + __float_as_uint(b);
  }
  const uint32_t off = 0x4B400000u * 0x1111u - 0x8888u;
  return (lo - off) | (hi - off) << 16;
}

}  // namespace kv4
}  // namespace msa
