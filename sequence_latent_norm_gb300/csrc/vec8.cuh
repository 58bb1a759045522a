// Eight (or one) neighbouring bf16 or fp32 channels as fp32 pairs.
#pragma once

#include "common.cuh"

namespace laga {

template <int V>
LAGA_DEVINL void load_vec(const float* p, float2 (&f)[(V + 1) / 2]) {
  if constexpr (V == 8) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
    const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    f[0] = make_float2(a.x, a.y); f[1] = make_float2(a.z, a.w);
    f[2] = make_float2(b.x, b.y); f[3] = make_float2(b.z, b.w);
  } else {
    f[0] = make_float2(*p, 0.f);
  }
}
template <int V>
LAGA_DEVINL void load_vec(const __nv_bfloat16* p, float2 (&f)[(V + 1) / 2]) {
  if constexpr (V == 8) {
    const uint4 w = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      f[k] = make_float2(__uint_as_float(u[k] << 16), __uint_as_float(u[k] & 0xffff0000u));
  } else {
    f[0] = make_float2(__bfloat162float(*p), 0.f);
  }
}
template <int V>
LAGA_DEVINL void store_vec(float* p, const float2 (&f)[(V + 1) / 2]) {
  if constexpr (V == 8) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
  } else {
    *p = f[0].x;
  }
}
template <int V>
LAGA_DEVINL void store_vec(__nv_bfloat16* p, const float2 (&f)[(V + 1) / 2]) {
  if constexpr (V == 8) {
    uint32_t u[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(f[k].x, f[k].y);
      u[k] = *reinterpret_cast<const uint32_t*>(&v);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
  } else {
    *p = __float2bfloat16_rn(f[0].x);
  }
}

// Vectors of 16 bytes (8 bf16 or 4 fp32) that stay packed until they are used.
template <typename T>
constexpr int vec16 = 16 / (int)sizeof(T);
LAGA_DEVINL void open16(const uint4& w, const float*, float2 (&f)[2]) {
  f[0] = make_float2(__uint_as_float(w.x), __uint_as_float(w.y));
  f[1] = make_float2(__uint_as_float(w.z), __uint_as_float(w.w));
}
LAGA_DEVINL void open16(const uint4& w, const __nv_bfloat16*, float2 (&f)[4]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    f[k] = make_float2(__uint_as_float(u[k] << 16), __uint_as_float(u[k] & 0xffff0000u));
}
LAGA_DEVINL uint4 close16(const float*, const float2 (&f)[2]) {
  return make_uint4(__float_as_uint(f[0].x), __float_as_uint(f[0].y), __float_as_uint(f[1].x),
                    __float_as_uint(f[1].y));
}
LAGA_DEVINL uint4 close16(const __nv_bfloat16*, const float2 (&f)[4]) {
  uint32_t u[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(f[k].x, f[k].y);
    u[k] = *reinterpret_cast<const uint32_t*>(&v);
  }
  return make_uint4(u[0], u[1], u[2], u[3]);
}

}  // namespace laga
