// The 8-bit block-scaled form of 32 columns, shared by the norm and the key-value cache.
#pragma once

#include "common.hpp"

namespace lora {

// The 8-bit form of the 32 columns that lanes 4i..4i+3 hold: the scale's biased
// exponent byte from the largest finite magnitude's bits (the least power of two
// with max <= 448 scale, so no finite value saturates), at least 1 (2^-126) and
// by the finite range at most 247, so that the scale and its reciprocal are
// normal fp32 numbers; then e4m3 codes, rounded to nearest even.  NaN and
// +-Inf become the NaN code.
__device__ __forceinline__ uint2 quantize8(const float* v, int& scale_byte) {
  float mx = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = fabsf(v[i]);
    mx = (a <= 3.4028234663852886e38f && a > mx) ? a : mx;
  }
  mx = fmaxf(mx, __shfl_xor(mx, 1, kWave));
  mx = fmaxf(mx, __shfl_xor(mx, 2, kWave));
  const int bits = __float_as_int(mx);
  const int b = max((bits >> 23) - 8 + ((bits & 0x7FFFFF) > 0x600000 ? 1 : 0), 1);
  scale_byte = b;
  const float mul = __int_as_float((254 - b) << 23);   // 2^(127 - b)
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) s[i] = v[i] * mul;
  int lo = __builtin_amdgcn_cvt_pk_fp8_f32(s[0], s[1], 0, false);
  lo = __builtin_amdgcn_cvt_pk_fp8_f32(s[2], s[3], lo, true);
  int hi = __builtin_amdgcn_cvt_pk_fp8_f32(s[4], s[5], 0, false);
  hi = __builtin_amdgcn_cvt_pk_fp8_f32(s[6], s[7], hi, true);
  return make_uint2((uint32_t)lo, (uint32_t)hi);
}

// The scale of an E8M0 byte from 1 to 254, 2^(b - 127).
__device__ __forceinline__ float e8m0(uint32_t b) { return __uint_as_float(b << 23); }

}  // namespace lora
