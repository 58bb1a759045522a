// Products of 8-bit operands (include/laga.h: laga_weight_pack, laga_mm8).
#include <algorithm>

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

// ------------------------------------------------------------------ product
constexpr int TM = 64, TN = 64, TK = 32;

template <typename T>
__global__ void __launch_bounds__(256)
    mm8_kernel(const uint8_t* __restrict__ a, const uint8_t* __restrict__ b,
               const int* __restrict__ start, T* __restrict__ y, int rows, int K, int N,
               int experts) {
  __shared__ float as[TK][TM + 1], bs[TK][TN + 1];
  __shared__ int seg[3];
  const int tid = threadIdx.x;
  if (tid == 0) {
    int left = blockIdx.y, e = 0, r0 = -1, r1 = 0;
    if (experts == 0) {
      r0 = left * TM;
      r1 = rows;
    } else {
      for (; e < experts; ++e) {
        const int s = start[e], t = min(start[e + 1], rows), n = (t - s + TM - 1) / TM;
        if (left < n) {
          r0 = s + left * TM;
          r1 = t;
          break;
        }
        left -= max(n, 0);
      }
    }
    seg[0] = e; seg[1] = r0; seg[2] = r1;
  }
  __syncthreads();
  const int e = seg[0], r0 = seg[1], r1 = seg[2];
  if (r0 < 0) return;
  const int n0 = blockIdx.x * TN, pitch = ck_pitch(K), cols = ck_cols(K);
  const uint8_t* bw = b + (long long)e * N * pitch;
  float acc[4][4] = {};
  const int tx = tid & 15, ty = tid >> 4;
  for (int k0 = 0; k0 < cols; k0 += TK) {
    const int i = tid >> 2, c = (tid & 3) * 8;
    float2 f[4];
    auto fetch = [&](const uint8_t* row) {
      const uint2 q = *reinterpret_cast<const uint2*>(row + k0 + c);
      const float unit = ck_unit(row[cols + k0 / CK_GROUP]);
      f[0] = ck_value2(q.x & 0xffffu, unit); f[1] = ck_value2(q.x >> 16, unit);
      f[2] = ck_value2(q.y & 0xffffu, unit); f[3] = ck_value2(q.y >> 16, unit);
    };
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = make_float2(0.f, 0.f);
    if (r0 + i < r1) fetch(a + (long long)(r0 + i) * pitch);
#pragma unroll
    for (int k = 0; k < 4; ++k) { as[c + 2 * k][i] = f[k].x; as[c + 2 * k + 1][i] = f[k].y; }
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = make_float2(0.f, 0.f);
    if (n0 + i < N) fetch(bw + (long long)(n0 + i) * pitch);
#pragma unroll
    for (int k = 0; k < 4; ++k) { bs[c + 2 * k][i] = f[k].x; bs[c + 2 * k + 1][i] = f[k].y; }
    __syncthreads();
#pragma unroll 8
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
      const int r = r0 + ty * 4 + p, n = n0 + tx * 4 + q;
      if (r < r1 && n < N) y[(long long)r * N + n] = from_f32<T>(acc[p][q]);
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

size_t mm8_ws_bytes(int rows, int K, int N, int experts, bool fp32) { return 0; }

cudaError_t launch_mm8(int rows, int K, int N, int experts, bool fp32, const void* a,
                       const void* b, const int* start, void* y, unsigned char* ws, int* err,
                       cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  const dim3 grid((N + TN - 1) / TN, (rows + TM - 1) / TM + experts);
  LaunchScope ls_("mm8", st);
  if (fp32)
    mm8_kernel<<<grid, 256, 0, st>>>(static_cast<const uint8_t*>(a),
                                     static_cast<const uint8_t*>(b), start,
                                     static_cast<float*>(y), rows, K, N, experts);
  else
    mm8_kernel<<<grid, 256, 0, st>>>(static_cast<const uint8_t*>(a),
                                     static_cast<const uint8_t*>(b), start,
                                     static_cast<__nv_bfloat16*>(y), rows, K, N, experts);
  return cudaGetLastError();
}

}  // namespace laga
