// The 8-bit checkpoint format (include/laga.h): e4m3 codes with one
// power-of-two scale per 128 channels of a row.
#pragma once

#include <cuda_fp8.h>
#include <stddef.h>

#include "common.cuh"

namespace laga {

constexpr int CK_GROUP = 128;                 // channels that share one scale
constexpr int CK_E_MIN = -117, CK_E_MAX = 119;
constexpr int CK_NAN = 255;                   // scale byte of a group with a non-finite value
constexpr int CK_MAX_D = 16384;
constexpr int CK_MAX_N = 1 << 20;            // columns of a weight gradient

// Bytes of a row's codes (whole groups), and of the whole row (scale bytes
// padded to 16, so that every row starts on a 16-byte boundary).
__host__ __device__ constexpr int ck_cols(int d) { return (d + CK_GROUP - 1) / CK_GROUP * CK_GROUP; }
__host__ __device__ constexpr int ck_pitch(int d) {
  return ck_cols(d) + (ck_cols(d) / CK_GROUP + 15) / 16 * 16;
}

// max(|a|, |b|) that keeps a NaN, for a group's maximum.
LAGA_DEVINL float ck_max(float a, float b) {
  float m;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(fabsf(a)), "f"(fabsf(b)));
  return m;
}

// Scale byte of a group whose maximum (ck_max) is m, and the factor 2^-e that
// its values are multiplied by before rounding.  With m = 1.f * 2^E: 448 =
// 1.75 * 2^8, so e is E - 8 for a significand up to 1.75 and E - 7 above.
// Both clamps keep 2^e and 2^-e normal fp32 and bf16 numbers.
LAGA_DEVINL int ck_scale(float m, float* inv) {
  const uint32_t u = __float_as_uint(m) & 0x7fffffffu;
  const int E = (int)(u >> 23) - 127;
  int e = E - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = min(max(e, CK_E_MIN), CK_E_MAX);
  *inv = __uint_as_float((uint32_t)(127 - e) << 23);
  return E == 128 ? CK_NAN : e + 127;   // infinity or NaN; the codes are then stored as zeros
}

// 2^e of a scale byte; NaN for a NaN group.
LAGA_DEVINL float ck_unit(uint32_t byte) {
  return byte == CK_NAN ? __uint_as_float(0x7fc00000u) : __uint_as_float(byte << 23);
}

// The codes of two values times 2^-e (low byte first).
LAGA_DEVINL uint32_t ck_code2(float2 v, float inv) {
  return __nv_cvt_float2_to_fp8x2(__fmul2_rn(v, make_float2(inv, inv)), __NV_SATFINITE,
                                  __NV_E4M3);
}

LAGA_DEVINL float2 ck_value2(uint32_t codes, float unit) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)codes, __NV_E4M3);
  return __fmul2_rn(__half22float2(__half2(h)), make_float2(unit, unit));
}

}  // namespace laga
