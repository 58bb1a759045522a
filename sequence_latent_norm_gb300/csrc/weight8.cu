// Weights in 8 bits (include/laga.h: laga_weight_pack).
#include "ckpt8.cuh"
#include "common.cuh"
#include "kernels.h"
#include "ops.h"

namespace laga {
namespace {

// ------------------------------------------------------------------ weights
// A block takes one 128 x 128 block of W: its maximum, its codes, and these as
// 128-byte pieces of the rows of W^T (fwd) and of W (bwd).
constexpr int WB = CK_GROUP, W_LD = WB + 4;

template <typename T>
__global__ void __launch_bounds__(256)
    weight_pack_kernel(const T* __restrict__ w, uint8_t* __restrict__ fwd,
                       uint8_t* __restrict__ bwd, int K, int N) {
  __shared__ uint8_t tile[WB * W_LD];
  __shared__ float part[8];
  const int nb = blockIdx.x, kb = blockIdx.y, e = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31;
  const T* src = w + (long long)e * K * N;
  const int c = tid & 127, r0 = tid >> 7;
  const bool in = nb * WB + c < N;
  float v[WB / 2], m = 0.f;
#pragma unroll
  for (int i = 0; i < WB / 2; ++i) {
    const int k = kb * WB + r0 + 2 * i;
    v[i] = in && k < K ? to_f32(src[(long long)k * N + nb * WB + c]) : 0.f;
    m = ck_max(m, v[i]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = ck_max(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) part[tid >> 5] = m;
  __syncthreads();
  m = part[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) m = ck_max(m, part[i]);
  float inv;
  const int s = ck_scale(m, &inv);
#pragma unroll
  for (int i = 0; i < WB / 2; i += 2) {
    const uint32_t q = s == CK_NAN ? 0u : ck_code2(make_float2(v[i], v[i + 1]), inv);
    tile[(r0 + 2 * i) * W_LD + c] = (uint8_t)q;
    tile[(r0 + 2 * i + 2) * W_LD + c] = (uint8_t)(q >> 8);
  }
  __syncthreads();
  // what a row gets: a word of codes a lane, its scale byte, and behind the
  // last group zeros
  const int pk = ck_pitch(K), pn = ck_pitch(N), ck = ck_cols(K), cn = ck_cols(N);
  auto finish = [&](uint8_t* row, int cols, int b, int pitch) {
    if (lane == 0) row[cols + b] = (uint8_t)s;
    if (b == cols / WB - 1)
      for (int i = cols + cols / WB + lane; i < pitch; i += 32) row[i] = 0;
  };
  for (int n = tid >> 5; n < WB && nb * WB + n < N; n += 8) {
    uint8_t* row = fwd + ((long long)e * N + nb * WB + n) * pk;
    uint32_t q = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) q |= (uint32_t)tile[(4 * lane + j) * W_LD + n] << (8 * j);
    reinterpret_cast<uint32_t*>(row + kb * WB)[lane] = q;
    finish(row, ck, kb, pk);
  }
  if (!bwd) return;
  for (int k = tid >> 5; k < WB && kb * WB + k < K; k += 8) {
    uint8_t* row = bwd + ((long long)e * K + kb * WB + k) * pn;
    reinterpret_cast<uint32_t*>(row + nb * WB)[lane] =
        *reinterpret_cast<const uint32_t*>(tile + k * W_LD + 4 * lane);
    finish(row, cn, nb, pn);
  }
}

}  // namespace

cudaError_t launch_weight_pack(int experts, int K, int N, bool fp32, const void* w, void* fwd,
                               void* bwd, cudaStream_t st) {
  const dim3 grid((N + WB - 1) / WB, (K + WB - 1) / WB, experts);
  LaunchScope ls_("weight_pack", st);
  if (fp32)
    weight_pack_kernel<<<grid, 256, 0, st>>>(static_cast<const float*>(w),
                                             static_cast<uint8_t*>(fwd),
                                             static_cast<uint8_t*>(bwd), K, N);
  else
    weight_pack_kernel<<<grid, 256, 0, st>>>(static_cast<const __nv_bfloat16*>(w),
                                             static_cast<uint8_t*>(fwd),
                                             static_cast<uint8_t*>(bwd), K, N);
  return cudaGetLastError();
}

}  // namespace laga
