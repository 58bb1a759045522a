// 8-bit checkpoints (include/laga.h: laga_ckpt_pack, laga_ckpt_unpack).
#include <algorithm>

#include "ckpt8.cuh"
#include "common.cuh"
#include "kernels.h"
#include "ops.h"

namespace laga {
namespace {

// Widths of a multiple of 8, where rows start on 16 bytes: a thread takes 8
// channels, 16 neighbouring threads a group, a block ROWS rows at a time, and
// issues UNROLL vectors' loads before it works on any.  Both kernels move 3
// bytes per bf16 element.  Unpacking does little else (16384 x 7168: 62 us with
// 4, 72 us with 1; 0.84 of the HBM rate); packing, with the group's maximum
// and the conversions, gains more from the warps that fewer registers allow
// (80 us with 1, 88 us with 2, 102 us with 4).
constexpr int ROWS = 8, PACK_UNROLL = 1, UNPACK_UNROLL = 4;

LAGA_DEVINL void load8(const float* p, float2 (&f)[4]) {
  const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
  const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
  f[0] = make_float2(a.x, a.y); f[1] = make_float2(a.z, a.w);
  f[2] = make_float2(b.x, b.y); f[3] = make_float2(b.z, b.w);
}
LAGA_DEVINL void load8(const __nv_bfloat16* p, float2 (&f)[4]) {
  const uint4 w = __ldcs(reinterpret_cast<const uint4*>(p));
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    f[k] = make_float2(__uint_as_float(u[k] << 16), __uint_as_float(u[k] & 0xffff0000u));
}
LAGA_DEVINL void store8(float* p, const float2 (&f)[4]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
}
LAGA_DEVINL void store8(__nv_bfloat16* p, const float2 (&f)[4]) {
  uint32_t u[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(f[k].x, f[k].y);
    u[k] = *reinterpret_cast<const uint32_t*>(&v);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}

template <typename T>
__global__ void __launch_bounds__(256) ckpt_pack8_kernel(const T* __restrict__ x, uint8_t* ck,
                                                         int rows, int d) {
  const int cols = ck_cols(d), vpr = cols / 8, pitch = ck_pitch(d);
  const int pad = pitch - cols - cols / CK_GROUP;
  for (long long r0 = (long long)blockIdx.x * ROWS; r0 < rows; r0 += (long long)gridDim.x * ROWS) {
    const int n = (int)min((long long)ROWS, rows - r0) * vpr;
    // whole warps go round, so that every lane of a group is there
    for (int i0 = threadIdx.x & ~31; i0 < n; i0 += 256 * PACK_UNROLL) {
      float2 f[PACK_UNROLL][4];
#pragma unroll
      for (int u = 0; u < PACK_UNROLL; ++u) {
        const int i = i0 + u * 256 + (threadIdx.x & 31);
        const int r = i / vpr, v = i - r * vpr;
#pragma unroll
        for (int k = 0; k < 4; ++k) f[u][k] = make_float2(0.f, 0.f);
        if (i < n && v * 8 < d) load8(x + (r0 + r) * d + v * 8, f[u]);
      }
#pragma unroll
      for (int u = 0; u < PACK_UNROLL; ++u) {
        const int i = i0 + u * 256 + (threadIdx.x & 31);
        const int r = i / vpr, v = i - r * vpr;
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) m = ck_max(ck_max(m, f[u][k].x), f[u][k].y);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m = ck_max(m, __shfl_xor_sync(0xffffffffu, m, o));
        float inv;
        const int s = ck_scale(m, &inv);
        if (i >= n) continue;
        uint8_t* row = ck + (r0 + r) * pitch;
        const uint32_t lo = ck_code2(f[u][0], inv) | ck_code2(f[u][1], inv) << 16;
        const uint32_t hi = ck_code2(f[u][2], inv) | ck_code2(f[u][3], inv) << 16;
        reinterpret_cast<uint2*>(row)[v] = s == CK_NAN ? make_uint2(0, 0) : make_uint2(lo, hi);
        if ((v & 15) == 0) row[cols + (v >> 4)] = (uint8_t)s;
        if (v < pad) row[cols + cols / CK_GROUP + v] = 0;
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(256) ckpt_unpack8_kernel(const uint8_t* __restrict__ ck, T* x,
                                                           int rows, int d) {
  const int cols = ck_cols(d), vpr = d / 8, pitch = ck_pitch(d);
  for (long long r0 = (long long)blockIdx.x * ROWS; r0 < rows; r0 += (long long)gridDim.x * ROWS) {
    const int n = (int)min((long long)ROWS, rows - r0) * vpr;
    for (int i0 = threadIdx.x; i0 < n; i0 += 256 * UNPACK_UNROLL) {
      uint2 q[UNPACK_UNROLL];
      uint32_t s[UNPACK_UNROLL];
#pragma unroll
      for (int u = 0; u < UNPACK_UNROLL; ++u) {
        const int i = i0 + u * 256, r = i / vpr, v = i - r * vpr;
        if (i < n) {
          const uint8_t* row = ck + (r0 + r) * pitch;
          q[u] = __ldcs(reinterpret_cast<const uint2*>(row) + v);
          s[u] = row[cols + (v >> 4)];
        }
      }
#pragma unroll
      for (int u = 0; u < UNPACK_UNROLL; ++u) {
        const int i = i0 + u * 256, r = i / vpr, v = i - r * vpr;
        if (i >= n) continue;
        const float unit = ck_unit(s[u]);
        const float2 f[4] = {ck_value2(q[u].x & 0xffffu, unit), ck_value2(q[u].x >> 16, unit),
                             ck_value2(q[u].y & 0xffffu, unit), ck_value2(q[u].y >> 16, unit)};
        store8(x + (r0 + r) * d + v * 8, f);
      }
    }
  }
}

// Other widths: one warp per 128-channel group, 4 channels a lane.
template <typename T>
__global__ void __launch_bounds__(256) ckpt_pack_kernel(const T* __restrict__ x, uint8_t* ck,
                                                        int rows, int d) {
  const int cols = ck_cols(d), groups = cols / CK_GROUP, pitch = ck_pitch(d);
  const int lane = threadIdx.x & 31;
  const long long n = (long long)rows * groups;
  for (long long w = blockIdx.x * 8LL + (threadIdx.x >> 5); w < n; w += gridDim.x * 8LL) {
    const long long r = w / groups;
    const int g = (int)(w % groups);
    uint8_t* row = ck + r * pitch;
    float t[4], m = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = g * CK_GROUP + 4 * lane + k;
      t[k] = c < d ? to_f32(x[r * d + c]) : 0.f;
      m = ck_max(m, t[k]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = ck_max(m, __shfl_xor_sync(0xffffffffu, m, o));
    float inv;
    const int s = ck_scale(m, &inv);
    const uint32_t q = ck_code2(make_float2(t[0], t[1]), inv) |
                       ck_code2(make_float2(t[2], t[3]), inv) << 16;
    *reinterpret_cast<uint32_t*>(row + g * CK_GROUP + 4 * lane) = s == CK_NAN ? 0u : q;
    if (lane == 0) row[cols + g] = (uint8_t)s;
    if (g == 0)
      for (int i = cols + groups + lane; i < pitch; i += 32) row[i] = 0;
  }
}

template <typename T>
__global__ void __launch_bounds__(256) ckpt_unpack_kernel(const uint8_t* __restrict__ ck, T* x,
                                                          int rows, int d) {
  const int cols = ck_cols(d), groups = cols / CK_GROUP, pitch = ck_pitch(d);
  const int lane = threadIdx.x & 31;
  const long long n = (long long)rows * groups;
  for (long long w = blockIdx.x * 8LL + (threadIdx.x >> 5); w < n; w += gridDim.x * 8LL) {
    const long long r = w / groups;
    const int g = (int)(w % groups);
    const uint8_t* row = ck + r * pitch;
    const float unit = ck_unit(row[cols + g]);
    const uint32_t q = *reinterpret_cast<const uint32_t*>(row + g * CK_GROUP + 4 * lane);
    const float2 a = ck_value2(q & 0xffffu, unit), b = ck_value2(q >> 16, unit);
    const float v[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = g * CK_GROUP + 4 * lane + k;
      if (c < d) x[r * d + c] = from_f32<T>(v[k]);
    }
  }
}

int row_grid(int rows) { return std::min((rows - 1) / ROWS + 1, 152 * 8); }

int warp_grid(int rows, int d) {
  const long long w = (long long)rows * (ck_cols(d) / CK_GROUP);
  return (int)std::min<long long>((w + 7) / 8, 152 * 8);
}

}  // namespace

cudaError_t launch_ckpt_pack(int rows, int d, bool fp32, const void* x, void* ck, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  LaunchScope ls_("ckpt_pack", st);
  if (d % 8 == 0 && fp32)
    ckpt_pack8_kernel<<<row_grid(rows), 256, 0, st>>>(static_cast<const float*>(x),
                                                      static_cast<uint8_t*>(ck), rows, d);
  else if (d % 8 == 0)
    ckpt_pack8_kernel<<<row_grid(rows), 256, 0, st>>>(static_cast<const __nv_bfloat16*>(x),
                                                      static_cast<uint8_t*>(ck), rows, d);
  else if (fp32)
    ckpt_pack_kernel<float><<<warp_grid(rows, d), 256, 0, st>>>(
        static_cast<const float*>(x), static_cast<uint8_t*>(ck), rows, d);
  else
    ckpt_pack_kernel<__nv_bfloat16><<<warp_grid(rows, d), 256, 0, st>>>(
        static_cast<const __nv_bfloat16*>(x), static_cast<uint8_t*>(ck), rows, d);
  return cudaGetLastError();
}

cudaError_t launch_ckpt_unpack(int rows, int d, bool fp32, const void* ck, void* x,
                               cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  LaunchScope ls_("ckpt_unpack", st);
  if (d % 8 == 0 && fp32)
    ckpt_unpack8_kernel<<<row_grid(rows), 256, 0, st>>>(static_cast<const uint8_t*>(ck),
                                                        static_cast<float*>(x), rows, d);
  else if (d % 8 == 0)
    ckpt_unpack8_kernel<<<row_grid(rows), 256, 0, st>>>(static_cast<const uint8_t*>(ck),
                                                        static_cast<__nv_bfloat16*>(x), rows, d);
  else if (fp32)
    ckpt_unpack_kernel<float><<<warp_grid(rows, d), 256, 0, st>>>(
        static_cast<const uint8_t*>(ck), static_cast<float*>(x), rows, d);
  else
    ckpt_unpack_kernel<__nv_bfloat16><<<warp_grid(rows, d), 256, 0, st>>>(
        static_cast<const uint8_t*>(ck), static_cast<__nv_bfloat16*>(x), rows, d);
  return cudaGetLastError();
}

}  // namespace laga
