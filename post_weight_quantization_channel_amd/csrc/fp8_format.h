// The 8-bit block format shared by the quantizer, the gated block's saved activations and the
// gradients that read them: e4m3 codes (largest finite value 448, no infinity, NaN 0x7F), one
// fp32 scale per block of 128 channels.
//
// The quantizer's scale is the power of two 2^e with the smallest e for which the block's largest
// magnitude is at most 448 2^e (e >= -126). Dividing by it is exact, so each code is the nearest
// e4m3 value of x / scale (ties to even) with a single rounding, and code times scale needs four
// significant bits: exact in bf16 and fp32. Against the scale max / 448 it gives up at most one
// binade at the bottom of the code's range (2^-9 2^e instead of 2^-9 max / 448), no precision
// above it.
#pragma once

#include "device_common.h"

namespace awq {

typedef int intx8 __attribute__((ext_vector_type(8)));

struct Fp8Scale {
  float scale;   // 2^e
  float inv;     // 2^-e
};

// amax: the block's largest finite magnitude. 2^e from its bits: 448 = 1.75 2^8, so with
// amax = 1.f 2^p the wanted e is p - 8 while 1.f <= 1.75 and p - 7 above. e lies in
// [-126, 120], so both 2^e and 2^-e are normal numbers. A block of zeros gets scale 1.
__device__ __forceinline__ Fp8Scale fp8_scale(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = (int)(u >> 23) - 127 - 8 + (((u & 0x7FFFFFu) > 0x600000u) ? 1 : 0);
  e = e < -126 ? -126 : e;
  Fp8Scale s;
  s.scale = u == 0u ? 1.0f : __uint_as_float((uint32_t)(127 + e) << 23);
  s.inv = u == 0u ? 1.0f : __uint_as_float((uint32_t)(127 - e) << 23);
  return s;
}

// Four values (each |v| <= 448) to four codes, the first in the low byte.
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
  return (uint32_t)r;
}

// The four values of a word of codes.
__device__ __forceinline__ void fp8_unpack4(uint32_t w, float (&v)[4]) {
  const auto lo = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, false);
  const auto hi = __builtin_amdgcn_cvt_pk_f32_fp8((int)w, true);
  v[0] = lo[0];
  v[1] = lo[1];
  v[2] = hi[0];
  v[3] = hi[1];
}

// Largest finite |v[t]| of eight values. Returns a bit per value that is an Inf or NaN: those are
// left out of the maximum, and fp8_pack8 gives them the NaN code.
__device__ __forceinline__ uint32_t fp8_absmax8(const float (&v)[8], float& amax) {
  uint32_t m = 0u, bad = 0u;
#pragma unroll
  for (int t = 0; t < 8; ++t) m = max(m, __float_as_uint(v[t]) & 0x7FFFFFFFu);
  if (m >= 0x7F800000u) {
    m = 0u;
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const uint32_t a = __float_as_uint(v[t]) & 0x7FFFFFFFu;
      if (a >= 0x7F800000u)
        bad |= 1u << t;
      else
        m = max(m, a);
    }
  }
  amax = __uint_as_float(m);
  return bad;
}

// The eight codes of v[t] / scale; 0x7F where `bad` (fp8_absmax8) has the value's bit set.
__device__ __forceinline__ uint2 fp8_pack8(const float (&v)[8], float inv, uint32_t bad) {
  uint2 p = make_uint2(fp8_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                       fp8_pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
  if (bad) {
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const uint32_t nan = 0x7Fu << (8 * t), keep = ~(0xFFu << (8 * t));
      if (bad >> t & 1u) p.x = (p.x & keep) | nan;
      if (bad >> (t + 4) & 1u) p.y = (p.y & keep) | nan;
    }
  }
  return p;
}

}  // namespace awq
