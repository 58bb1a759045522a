// Weight gradient by expert (include/laga.h: laga_experts_dw).
#include <algorithm>

#include "ckpt8.cuh"
#include "common.cuh"
#include "kernels.h"
#include "ops.h"

namespace laga {
namespace {

constexpr int TM = 64, TN = 64, TK = 16;

template <typename T>
__global__ void __launch_bounds__(256)
    experts_dw_kernel(const uint8_t* __restrict__ ck, const T* __restrict__ dy,
                      const float* __restrict__ gamma, const int* __restrict__ start,
                      float* __restrict__ dw, int rows, int d, int n) {
  __shared__ float as[TK][TM + 1], bs[TK][TN + 1];
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int n0 = blockIdx.x * TN, d0 = blockIdx.y * TM, e = blockIdx.z;
  const int r1 = min(rows, start[e + 1]), pitch = ck_pitch(d), cols = ck_cols(d);
  float acc[4][4] = {};
  for (int r0 = start[e]; r0 < r1; r0 += TK) {
    for (int i = tid; i < TK * TM; i += 256) {
      const int r = r0 + i / TM, c = d0 + i % TM;
      float v = 0.f;
      if (r < r1 && c < d) {
        const uint8_t* row = ck + (long long)r * pitch;
        v = ck_value2(row[c], ck_unit(row[cols + c / CK_GROUP])).x;
      }
      as[i / TM][i % TM] = v;
    }
    for (int i = tid; i < TK * TN; i += 256) {
      const int r = r0 + i / TN, c = n0 + i % TN;
      bs[i / TN][i % TN] = r < r1 && c < n ? to_f32(dy[(long long)r * n + c]) : 0.f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < TK; ++k)
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int q = 0; q < 4; ++q) acc[p][q] += as[k][ty * 4 + p] * bs[k][tx * 4 + q];
    __syncthreads();
  }
#pragma unroll
  for (int p = 0; p < 4; ++p)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int i = d0 + ty * 4 + p, j = n0 + tx * 4 + q;
      if (i < d && j < n)
        dw[((long long)e * d + i) * n + j] = gamma ? gamma[i] * acc[p][q] : acc[p][q];
    }
}

}  // namespace

size_t experts_dw_ws_bytes(int rows, int d, int n, int experts, bool fp32) { return 0; }

cudaError_t launch_experts_dw(int rows, int d, int n, int experts, bool fp32, const void* ck,
                              const void* dy, const float* gamma, const int* start, float* dw,
                              unsigned char* ws, int* err, cudaStream_t st) {
  if (rows == 0) return cudaMemsetAsync(dw, 0, (size_t)experts * d * n * 4, st);
  const dim3 grid((n + TN - 1) / TN, (d + TM - 1) / TM, experts);
  LaunchScope ls_("experts_dw", st);
  if (fp32)
    experts_dw_kernel<<<grid, 256, 0, st>>>(static_cast<const uint8_t*>(ck),
                                            static_cast<const float*>(dy), gamma, start, dw, rows,
                                            d, n);
  else
    experts_dw_kernel<<<grid, 256, 0, st>>>(static_cast<const uint8_t*>(ck),
                                            static_cast<const __nv_bfloat16*>(dy), gamma, start,
                                            dw, rows, d, n);
  return cudaGetLastError();
}

}  // namespace laga
