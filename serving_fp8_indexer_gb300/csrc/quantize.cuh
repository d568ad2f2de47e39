// What the operators that write low-precision rows share: the scale of a block
// of values, the quotient by it, and the 4-bit cache row.
#pragma once
#include "ptx.cuh"

namespace smla {

constexpr float kE4m3Max = 448.f;

SMLA_DEVICE_INLINE float finite_abs(float v) {
  const float a = fabsf(v);
  return a < INFINITY ? a : 0.f;  // false for NaN
}
// The scale that maps `amax` to e4m3's largest value; 1 for an all-zero
// block, and never below the smallest normal number (so that x / scale and
// byte * scale stay finite).
SMLA_DEVICE_INLINE float scale_of(float amax, float top = kE4m3Max) {
  return amax > 0.f ? fmaxf(amax / top, 1.17549435e-38f) : 1.f;
}

// v / scale, rounded once: the product with the rounded reciprocal is off by up to
// 1.5 units in the last place, and a quotient on the border between two bytes then
// fell to the wrong side.  One step with the exact remainder mends that (Markstein,
// IBM J. Res. Dev. 34, 1990): 12 117 block-scaled rows 13.0 -> 13.75 us, by a
// division each 15.3.  (The remainder is exact while scale >= 2^-100.)  Without one
// to speak of, as for infinities, NaN and zeros, the product stands.
SMLA_DEVICE_INLINE float quotient(float v, float scale, float inv) {
  const float q = v * inv;
  const float r = fmaf(-q, scale, v);
  return fabsf(r) > 0.f ? fmaf(r, inv, q) : q;
}

// ------------------------------------------------------------ the 4-bit cache row
// 576 values in 320 bytes: 288 bytes of e2m1 codes (the even column in the low
// half), 18 bytes of shifts (four bits for each 16 columns, the even block in the
// low half), two zero bytes, the row's scale in f32, eight zero bytes.
//   value = e2m1 * 2^(6 - shift) * scale
// scale = largest magnitude / 384, so the row's largest value is 6 * 2^6 units, and
// shift (0..14) is the largest that keeps the block's within 6 code units: 14 for a
// block of zeros.  15 is never written; readers take such a block as zeros whatever
// its codes.  e2m1 * 2^(6 - shift) is an e4m3 number for every
// code and shift (0.5 * 2^-8 is e4m3's smallest): attention reads the row on the
// FP8 pipe as it is held, with the scale by the row.
constexpr int kFp4Row = 320, kFp4Shifts = 288, kFp4Scale = 308, kFp4Blocks = 36;
constexpr float kFp4Top = 384.f;
constexpr int kFp4MaxShift = 14;

// Shift of a block whose largest finite magnitude is `top`, of a row whose is
// `most`: the largest k in 0..14 with top * 2^k <= most.
SMLA_DEVICE_INLINE int fp4_shift(float top, float most) {
  if (top == 0.f) return kFp4MaxShift;
  if (most < 0x1p-60f) {  // (their exponents are read as those of normal numbers)
    top *= 0x1p60f;
    most *= 0x1p60f;
  }
  const int et = static_cast<int>(__float_as_uint(top) >> 23), em = static_cast<int>(__float_as_uint(most) >> 23);
  int k = min(em - et, kFp4MaxShift);
  if (k > 0 && top * __uint_as_float(static_cast<uint32_t>(127 + k) << 23) > most) --k;
  return max(k, 0);
}

// Eight floats -> eight e2m1 codes (nearest even, past +-6 become +-6).
SMLA_DEVICE_INLINE uint32_t pack_e2m1x8(const float (&x)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
  return r;
}

// Table entry of a shift: the e4m3 bytes of the magnitudes 0, 0.5, 1, 1.5 (x) and
// 2, 3, 4, 6 (y) times 2^(6 - shift); zeros for shift 15.
SMLA_DEVICE_INLINE uint2 fp4_table_entry(int shift) {
  if (shift > kFp4MaxShift) return make_uint2(0u, 0u);
  const float u = __uint_as_float(static_cast<uint32_t>(127 + 6 - shift) << 23);
  return make_uint2(static_cast<uint32_t>(f32x2_to_e4m3x2(0.f, 0.5f * u)) |
                        static_cast<uint32_t>(f32x2_to_e4m3x2(u, 1.5f * u)) << 16,
                    static_cast<uint32_t>(f32x2_to_e4m3x2(2.f * u, 3.f * u)) |
                        static_cast<uint32_t>(f32x2_to_e4m3x2(4.f * u, 6.f * u)) << 16);
}
// Eight codes -> eight e4m3 bytes, by the entry t of their block's shift: each
// code's three magnitude bits select a byte, then the signs are put in.
SMLA_DEVICE_INLINE uint2 fp4x8_to_e4m3x8(uint32_t w, uint2 t) {
  const uint32_t m = w & 0x77777777u, x = w << 4;
  const uint32_t lo = __byte_perm(t.x, t.y, m), hi = __byte_perm(t.x, t.y, m >> 16);
  return make_uint2(lo | (__byte_perm(w, x, 0x1504) & 0x80808080u), hi | (__byte_perm(w, x, 0x3726) & 0x80808080u));
}

}  // namespace smla
