// Weights in 8 bits (include/laga.h: laga_weight_pack).
#include "ckpt8.cuh"
#include "common.cuh"
#include "kernels.h"
#include "ops.h"
#include "vec8.cuh"

namespace laga {
namespace {

// A block takes one 128 x 128 block of W: its maximum, its codes, and these as
// 128-byte pieces of the rows of W^T (fwd) and of W (bwd).  A thread loads 8
// columns of 8 rows.  The codes are turned in shared memory in words of 4: word w
// of row r sits at w ^ (r / 4), so that reading rows 4 l .. 4 l + 3 of one word by
// lane l, like writing, meets every bank once.  It moves 0.7 of what HBM could at
// 32 x 7168 x 4096 (799 us): every row of a block ends in a scale byte, which one lane
// stores, and the bf16 kernel spills 64 bytes at its 64 registers.  (7168 x 1536
// bf16: 10 us within a graph.)
// The values stay as they were loaded until they are coded, so that four blocks of
// bf16 weights fit an SM (32 x 7168 x 4096: 881 us as floats, three blocks).
constexpr int WB = CK_GROUP;

template <typename T>
struct Eight;   // eight neighbouring values
template <>
struct Eight<float> {
  float2 v[4];
  LAGA_DEVINL float2 at(int j) const { return v[j]; }
  LAGA_DEVINL void load(const float* p) { load_vec<8>(p, v); }
  LAGA_DEVINL void set(int j, float a, float b) { v[j] = make_float2(a, b); }
};
template <>
struct Eight<__nv_bfloat16> {
  uint32_t v[4];
  LAGA_DEVINL float2 at(int j) const {
    return make_float2(__uint_as_float(v[j] << 16), __uint_as_float(v[j] & 0xffff0000u));
  }
  LAGA_DEVINL void load(const __nv_bfloat16* p) {
    const uint4 w = __ldcs(reinterpret_cast<const uint4*>(p));
    v[0] = w.x; v[1] = w.y; v[2] = w.z; v[3] = w.w;
  }
  LAGA_DEVINL void set(int j, float a, float b) {   // (bf16 values: nothing is rounded)
    v[j] = __float_as_uint(a) >> 16 | (__float_as_uint(b) & 0xffff0000u);
  }
};

template <typename T, int V>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 4 : 3)
    weight_pack_kernel(const T* __restrict__ w, uint8_t* __restrict__ fwd,
                       uint8_t* __restrict__ bwd, int K, int N) {
  __shared__ uint32_t tile[WB][WB / 4];
  __shared__ float part[8];
  const int nb = blockIdx.x, kb = blockIdx.y, e = blockIdx.z;
  const int tid = threadIdx.x, lane = tid & 31;
  const T* src = w + (long long)e * K * N;
  const int c = (tid & 15) * 8, r0 = tid >> 4;
  Eight<T> v[8];
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int k = kb * WB + r0 + 16 * i, n = nb * WB + c;
    const T* p = src + (long long)k * N + n;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[i].set(j, 0.f, 0.f);
    if (k < K) {
      if constexpr (V == 8) {
        if (n < N) v[i].load(p);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[i].set(j, n + 2 * j < N ? to_f32(p[2 * j]) : 0.f,
                   n + 2 * j + 1 < N ? to_f32(p[2 * j + 1]) : 0.f);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = v[i].at(j);
      m = ck_max(ck_max(m, f.x), f.y);
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
  for (int i = 0; i < 8; ++i) {
    const int r = r0 + 16 * i, x = r >> 2;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t q = ck_code2(v[i].at(2 * h), inv) | ck_code2(v[i].at(2 * h + 1), inv) << 16;
      tile[r][(c / 4 + h) ^ x] = s == CK_NAN ? 0u : q;
    }
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
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    // 4 rows x 4 columns of codes, turned
    const int cw = (tid >> 5) + 8 * i;
    uint32_t q[4], o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = tile[4 * lane + j][cw ^ lane];
    const uint32_t a = __byte_perm(q[0], q[1], 0x5140), b = __byte_perm(q[2], q[3], 0x5140);
    const uint32_t d = __byte_perm(q[0], q[1], 0x7362), g = __byte_perm(q[2], q[3], 0x7362);
    o[0] = __byte_perm(a, b, 0x5410);
    o[1] = __byte_perm(a, b, 0x7632);
    o[2] = __byte_perm(d, g, 0x5410);
    o[3] = __byte_perm(d, g, 0x7632);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int n = nb * WB + 4 * cw + j;
      if (n >= N) break;
      uint8_t* row = fwd + ((long long)e * N + n) * pk;
      reinterpret_cast<uint32_t*>(row + kb * WB)[lane] = o[j];
      finish(row, ck, kb, pk);
    }
  }
  if (!bwd) return;
  for (int k = tid >> 5; k < WB && kb * WB + k < K; k += 8) {
    uint8_t* row = bwd + ((long long)e * K + kb * WB + k) * pn;
    reinterpret_cast<uint32_t*>(row + nb * WB)[lane] = tile[k][lane ^ (k >> 2)];
    finish(row, cn, nb, pn);
  }
}

}  // namespace

cudaError_t launch_weight_pack(int experts, int K, int N, bool fp32, const void* w, void* fwd,
                               void* bwd, cudaStream_t st) {
  const dim3 grid((N + WB - 1) / WB, (K + WB - 1) / WB, experts);
  uint8_t *f = static_cast<uint8_t*>(fwd), *b = static_cast<uint8_t*>(bwd);
  LaunchScope ls_("weight_pack", st);
  if (fp32) {
    auto k = N % 8 == 0 ? weight_pack_kernel<float, 8> : weight_pack_kernel<float, 1>;
    k<<<grid, 256, 0, st>>>(static_cast<const float*>(w), f, b, K, N);
  } else {
    auto k = N % 8 == 0 ? weight_pack_kernel<__nv_bfloat16, 8>
                        : weight_pack_kernel<__nv_bfloat16, 1>;
    k<<<grid, 256, 0, st>>>(static_cast<const __nv_bfloat16*>(w), f, b, K, N);
  }
  return cudaGetLastError();
}

}  // namespace laga
