// Rows of an 8-bit cache: D codes (e4m3 or e5m2) and one scale 2^e of a token
// and KV head, kept as the byte e + 127.
//
// A power of two as the scale: code * 2^e is a bf16 number exactly, a score is
// multiplied by it without a rounding, a value's scale joins the exponent of its
// probability, and it takes a byte where an fp32 scale takes four (3 % of a row
// of 128).  What it costs is at most one bit of the codes' range, none of their
// precision: e is the least at which no code exceeds the format's largest value
// (448 or 57344, both 1.75 * 2^x).
#pragma once
#include <cstdint>

#include "fa_paged.cuh"

namespace fa {

constexpr int kLeastExp = -80;          // of a scale: 2^31 times 2^(15 - e), a softmax's sum (fa_decode8.cuh), stays an fp32 number
constexpr uint32_t kScaleNone = 255;    // the scale byte of a row that was not finite

template <bool E5M2>
__device__ __forceinline__ uint32_t codes_f16x2(uint32_t two) {   // two codes in bits 0-15, exactly
  uint32_t r;
  if constexpr (E5M2)
    asm("{\n .reg .b16 t;\n cvt.u16.u32 t, %1;\n cvt.rn.f16x2.e5m2x2 %0, t;\n}" : "=r"(r) : "r"(two));
  else
    asm("{\n .reg .b16 t;\n cvt.u16.u32 t, %1;\n cvt.rn.f16x2.e4m3x2 %0, t;\n}" : "=r"(r) : "r"(two));
  return r;
}
template <bool E5M2>
__device__ __forceinline__ uint32_t codes_of(float a, float b, float c, float d) {   // to the nearest codes, ties to even
  uint32_t r;
  if constexpr (E5M2)
    asm("{\n .reg .b16 l, h;\n cvt.rn.satfinite.e5m2x2.f32 l, %2, %1;\n cvt.rn.satfinite.e5m2x2.f32 h, %4, %3;\n mov.b32 %0, {l, h};\n}"
        : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
  else
    asm("{\n .reg .b16 l, h;\n cvt.rn.satfinite.e4m3x2.f32 l, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 h, %4, %3;\n mov.b32 %0, {l, h};\n}"
        : "=r"(r) : "f"(a), "f"(b), "f"(c), "f"(d));
  return r;
}
// the largest magnitude of three, NaN where one of them is
__device__ __forceinline__ float max3_abs_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// 2^e from the scale byte e + 127 (infinity from kScaleNone)
__device__ __forceinline__ float scale_of(uint32_t byte) { return __uint_as_float(byte << 23); }

// The codes of a row that L neighbouring lanes hold, 16 channels each, and its scale byte.  A row that
// is not finite becomes NaN (scale byte 255) and is reported: no code stands for an infinity.
template <int L>
__device__ __forceinline__ uint32_t quantise_row(const float (&a)[8], const float (&d)[8], int e5m2, uint2& qa,
                                                 uint2& qd, int* status) {
  float t0 = max3_abs_nan(a[0], a[1], a[2]), t1 = max3_abs_nan(d[0], d[1], d[2]);
  t0 = max3_abs_nan(t0, a[3], a[4]), t1 = max3_abs_nan(t1, d[3], d[4]);
  t0 = max3_abs_nan(t0, a[5], a[6]), t1 = max3_abs_nan(t1, d[5], d[6]);
  uint32_t top = __float_as_uint(max3_abs_nan(max3_abs_nan(t0, a[7], d[7]), t1, t1));
  const unsigned lane = threadIdx.x & 31;
  const unsigned row = ((1u << L) - 1u) << (lane & ~(unsigned)(L - 1));   // (rows of a warp may be on their own)
#pragma unroll
  for (int m = 1; m < L; m <<= 1) top = max(top, __shfl_xor_sync(row, top, m));   // (by its bits NaN is the largest)
  if (top >= 0x7F800000u) {
    qa = qd = make_uint2(0, 0);
    if ((lane & (L - 1)) == 0) atomicOr(status, fa_host::kStatusRange);
    return kScaleNone;
  }
  // the largest is m 2^x, 1 <= m < 2: it fits 1.75 * 2^(8 or 15) at e = x - (8 or 15), one more where m > 1.75
  // (no more than keeps the largest code an fp32 and bf16 number; there it saturates)
  const int fit = e5m2 ? 15 : 8;
  int e = (int)((top + 0x1FFFFFu) >> 23) - 127 - fit;      // (0x1FFFFF carries a mantissa above 0x600000)
  e = min(max(e, kLeastExp), 127 - fit);
  const float f = __uint_as_float((uint32_t)(127 - e) << 23);
  float x[8], y[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) x[j] = a[j] * f, y[j] = d[j] * f;
  if (e5m2) {
    qa = make_uint2(codes_of<true>(x[0], x[1], x[2], x[3]), codes_of<true>(x[4], x[5], x[6], x[7]));
    qd = make_uint2(codes_of<true>(y[0], y[1], y[2], y[3]), codes_of<true>(y[4], y[5], y[6], y[7]));
  } else {
    qa = make_uint2(codes_of<false>(x[0], x[1], x[2], x[3]), codes_of<false>(x[4], x[5], x[6], x[7]));
    qd = make_uint2(codes_of<false>(y[0], y[1], y[2], y[3]), codes_of<false>(y[4], y[5], y[6], y[7]));
  }
  return (uint32_t)(e + 127);
}

// The cache type's numbers around the eight values that codes stand for: a bf16 is the value itself, of
// fp16 (too narrow for some) the next below and above.
template <bool BF16, bool E5M2>
__device__ __forceinline__ void stored_bounds(uint2 codes, uint32_t scale, uint4& lo, uint4& hi) {
  const float f = scale_of(scale);
  uint32_t l[4], h[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t two = (j < 2 ? codes.x : codes.y) >> (16 * (j & 1));
    const uint32_t x = codes_f16x2<E5M2>(two);
    const float x0 = f16_lo_to_f32(x) * f, x1 = f16_hi_to_f32(x) * f;
    if constexpr (BF16) {
      l[j] = h[j] = pack_bf16x2(x0, x1);
    } else {
      uint16_t r0, r1;
      asm("cvt.rm.f16.f32 %0, %1;" : "=h"(r0) : "f"(x0));
      asm("cvt.rm.f16.f32 %0, %1;" : "=h"(r1) : "f"(x1));
      l[j] = r0 | (uint32_t)r1 << 16;
      asm("cvt.rp.f16.f32 %0, %1;" : "=h"(r0) : "f"(x0));
      asm("cvt.rp.f16.f32 %0, %1;" : "=h"(r1) : "f"(x1));
      h[j] = r0 | (uint32_t)r1 << 16;
    }
  }
  lo = make_uint4(l[0], l[1], l[2], l[3]);
  hi = make_uint4(h[0], h[1], h[2], h[3]);
}

// Eight codes as the cache's type, rounded once (exact in bf16).
template <bool BF16, bool E5M2>
__device__ __forceinline__ uint4 read_codes(uint2 codes, float f) {
  float x[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t two = (j < 2 ? codes.x : codes.y) >> (16 * (j & 1));
    const uint32_t h = codes_f16x2<E5M2>(two);
    x[2 * j] = f16_lo_to_f32(h) * f;
    x[2 * j + 1] = f16_hi_to_f32(h) * f;
  }
  return pack8<BF16>(x);
}

}  // namespace fa
