// 8-bit checkpoints (include/laga.h: laga_ckpt_pack, laga_ckpt_unpack).
#include <algorithm>

#include "ckpt8.cuh"
#include "common.cuh"
#include "kernels.h"
#include "ops.h"

namespace laga {
namespace {

// One warp per 128-channel group, 4 channels a lane.
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

int warp_grid(int rows, int d) {
  const long long w = (long long)rows * (ck_cols(d) / CK_GROUP);
  return (int)std::min<long long>((w + 7) / 8, 152 * 8);
}

}  // namespace

cudaError_t launch_ckpt_pack(int rows, int d, bool fp32, const void* x, void* ck, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  LaunchScope ls_("ckpt_pack", st);
  if (fp32)
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
  if (fp32)
    ckpt_unpack_kernel<float><<<warp_grid(rows, d), 256, 0, st>>>(
        static_cast<const uint8_t*>(ck), static_cast<float*>(x), rows, d);
  else
    ckpt_unpack_kernel<__nv_bfloat16><<<warp_grid(rows, d), 256, 0, st>>>(
        static_cast<const uint8_t*>(ck), static_cast<__nv_bfloat16*>(x), rows, d);
  return cudaGetLastError();
}

}  // namespace laga
