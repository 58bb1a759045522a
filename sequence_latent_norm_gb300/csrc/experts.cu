// Rows to experts and back, and the experts' gated activation (include/laga.h:
// laga_spread8, laga_combine_*, laga_swiglu_*).  All of it is bound by HBM.
#include <algorithm>

#include "ckpt8.cuh"
#include "common.cuh"
#include "kernels.h"
#include "ops.h"
#include "vec8.cuh"

namespace laga {
namespace {

// ------------------------------------------------------------------ rows
// A warp copies one row of codes, 16 bytes a lane.
__global__ void __launch_bounds__(256)
    spread8_kernel(const uint8_t* __restrict__ ck, const int* __restrict__ pair,
                   const int* __restrict__ end, uint8_t* __restrict__ out, int rows, int tokens,
                   int top_k, int pitch) {
  const int lane = threadIdx.x & 31, vecs = pitch / 16;
  const int n = min(rows, *end);
  for (long long r = blockIdx.x * 8LL + (threadIdx.x >> 5); r < n; r += gridDim.x * 8LL) {
    const int q = pair[r], t = q / top_k;
    uint4* dst = reinterpret_cast<uint4*>(out + r * pitch);
    if (q < 0 || t >= tokens) {
      for (int v = lane; v < vecs; v += 32) dst[v] = make_uint4(0, 0, 0, 0);
      continue;
    }
    const uint4* src = reinterpret_cast<const uint4*>(ck + (long long)t * pitch);
    for (int v = lane; v < vecs; v += 32) dst[v] = src[v];
  }
}

// out_t = sum_j w_tj y[row_tj]: a thread V channels of a token.
template <typename T, int V>
__global__ void __launch_bounds__(256)
    combine_kernel(const T* __restrict__ y, const float* __restrict__ weight,
                   const int* __restrict__ row, T* __restrict__ out, int tokens, int top_k,
                   int rows, int d) {
  const int vecs = d / V;
  const long long n = (long long)tokens * vecs;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < n; i += gridDim.x * 256LL) {
    const long long t = i / vecs;
    const int c = (int)(i - t * vecs) * V;
    float2 acc[(V + 1) / 2];
#pragma unroll
    for (int k = 0; k < (V + 1) / 2; ++k) acc[k] = make_float2(0.f, 0.f);
    for (int j = 0; j < top_k; ++j) {
      const int r = row[t * top_k + j];
      if (r < 0 || r >= rows) continue;
      const float w = weight ? weight[t * top_k + j] : 1.f;
      float2 f[(V + 1) / 2];
      load_vec<V>(y + (long long)r * d + c, f);
#pragma unroll
      for (int k = 0; k < (V + 1) / 2; ++k) acc[k] = __ffma2_rn(f[k], make_float2(w, w), acc[k]);
    }
    store_vec<V>(out + t * d + c, acc);
  }
}

// dy[row_tj] = w_tj dout_t, dw_tj = <dout_t, y[row_tj]>: a block a token, its
// choices one after the other; then the rows that no pair has, as zeros.
template <typename T, int V>
__global__ void __launch_bounds__(256)
    combine_bwd_kernel(const T* __restrict__ dout, const T* __restrict__ y,
                       const float* __restrict__ weight, const int* __restrict__ row,
                       const int* __restrict__ pair, const int* __restrict__ end,
                       T* __restrict__ dy, float* __restrict__ dweight, int tokens, int top_k,
                       int rows, int d) {
  __shared__ float part[8];
  const int vecs = d / V, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  for (long long t = blockIdx.x; t < tokens; t += gridDim.x) {
    for (int j = 0; j < top_k; ++j) {
      const int r = row[t * top_k + j];
      float dot = 0.f;
      if (r >= 0 && r < rows) {
        const float w = weight ? weight[t * top_k + j] : 1.f;
        for (int v = threadIdx.x; v < vecs; v += 256) {
          float2 g[(V + 1) / 2], f[(V + 1) / 2];
          load_vec<V>(dout + t * d + v * V, g);
          if (y) {
            load_vec<V>(y + (long long)r * d + v * V, f);
#pragma unroll
            for (int k = 0; k < (V + 1) / 2; ++k) dot += g[k].x * f[k].x + g[k].y * f[k].y;
          }
#pragma unroll
          for (int k = 0; k < (V + 1) / 2; ++k) g[k] = __fmul2_rn(g[k], make_float2(w, w));
          store_vec<V>(dy + (long long)r * d + v * V, g);
        }
      }
      if (!dweight) continue;
      dot = warp_sum(dot);
      if (lane == 0) part[warp] = dot;
      __syncthreads();
      if (threadIdx.x == 0) {
        float s = 0.f;
        for (int k = 0; k < 8; ++k) s += part[k];
        dweight[t * top_k + j] = s;
      }
      __syncthreads();
    }
  }
  const int n = rows > 0 ? min(rows, *end) : 0;
  for (long long r = blockIdx.x; r < n; r += gridDim.x)
    if (pair[r] < 0)
      for (int c = threadIdx.x; c < d; c += 256) dy[r * d + c] = from_f32<T>(0.f);
}

// ------------------------------------------------------------------ activation
LAGA_DEVINL float sigmoid_of(float x) { return 1.f / (1.f + expf(-x)); }

// a = silu(g) u of 4 channels a lane, a warp one group of 128.
template <typename T>
__global__ void __launch_bounds__(256)
    swiglu_kernel(const T* __restrict__ gu, uint8_t* __restrict__ ck, const int* __restrict__ end,
                  int rows, int f) {
  const int cols = ck_cols(f), groups = cols / CK_GROUP, pitch = ck_pitch(f);
  const int lane = threadIdx.x & 31;
  const long long n = (long long)(end ? min(rows, *end) : rows) * groups;
  for (long long w = blockIdx.x * 8LL + (threadIdx.x >> 5); w < n; w += gridDim.x * 8LL) {
    const long long r = w / groups;
    const int g = (int)(w % groups);
    uint8_t* row = ck + r * pitch;
    const T* src = gu + r * 2 * f;
    float t[4], m = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = g * CK_GROUP + 4 * lane + k;
      t[k] = 0.f;
      if (c < f) {
        const float x = to_f32(src[c]);
        t[k] = x * sigmoid_of(x) * to_f32(src[f + c]);
      }
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

// dg = da u sigma (1 + g (1 - sigma)), du = da g sigma.
template <typename T>
__global__ void __launch_bounds__(256)
    swiglu_bwd_kernel(const T* __restrict__ gu, const T* __restrict__ da, T* __restrict__ dgu,
                      const int* __restrict__ end, int rows, int f) {
  const long long n = (long long)(end ? min(rows, *end) : rows) * f;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < n; i += gridDim.x * 256LL) {
    const long long r = i / f;
    const int c = (int)(i - r * f);
    const long long o = r * 2 * f + c;
    const float g = to_f32(gu[o]), u = to_f32(gu[o + f]), d = to_f32(da[i]);
    const float sig = sigmoid_of(g);
    dgu[o] = from_f32<T>(d * u * sig * (1.f + g * sigmoid_of(-g)));
    dgu[o + f] = from_f32<T>(d * g * sig);
  }
}

int grid_for(long long blocks, int most) { return (int)std::max<long long>(1, std::min<long long>(blocks, most)); }

template <typename T>
cudaError_t combine_t(int tokens, int top_k, int rows, int d, const void* y, const float* weight,
                      const int* row, void* out, cudaStream_t st) {
  LaunchScope ls_("combine", st);
  const T* src = static_cast<const T*>(y);
  if (d % 8 == 0) {
    const int grid = grid_for(((long long)tokens * (d / 8) + 255) / 256, 152 * 8);
    combine_kernel<T, 8><<<grid, 256, 0, st>>>(src, weight, row, static_cast<T*>(out), tokens,
                                               top_k, rows, d);
  } else {
    const int grid = grid_for(((long long)tokens * d + 255) / 256, 152 * 8);
    combine_kernel<T, 1><<<grid, 256, 0, st>>>(src, weight, row, static_cast<T*>(out), tokens,
                                               top_k, rows, d);
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t combine_bwd_t(int tokens, int top_k, int rows, int d, const void* dout, const void* y,
                          const float* weight, const int* row, const int* pair, const int* end,
                          void* dy, float* dweight, cudaStream_t st) {
  LaunchScope ls_("combine_bwd", st);
  const int grid = grid_for(std::max(tokens, 1), 152 * 8);
  const T *g = static_cast<const T*>(dout), *f = static_cast<const T*>(y);
  if (d % 8 == 0)
    combine_bwd_kernel<T, 8><<<grid, 256, 0, st>>>(g, f, weight, row, pair, end,
                                                   static_cast<T*>(dy), dweight, tokens, top_k,
                                                   rows, d);
  else
    combine_bwd_kernel<T, 1><<<grid, 256, 0, st>>>(g, f, weight, row, pair, end,
                                                   static_cast<T*>(dy), dweight, tokens, top_k,
                                                   rows, d);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_spread8(int rows, int tokens, int top_k, int d, const void* ck, const int* pair,
                           const int* end, void* out, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  LaunchScope ls_("spread8", st);
  spread8_kernel<<<grid_for(((long long)rows + 7) / 8, 152 * 8), 256, 0, st>>>(
      static_cast<const uint8_t*>(ck), pair, end, static_cast<uint8_t*>(out), rows, tokens, top_k,
      ck_pitch(d));
  return cudaGetLastError();
}

cudaError_t launch_combine_fwd(int tokens, int top_k, int rows, int d, bool fp32, const void* y,
                               const float* weight, const int* row, void* out, cudaStream_t st) {
  if (tokens == 0) return cudaSuccess;
  return fp32 ? combine_t<float>(tokens, top_k, rows, d, y, weight, row, out, st)
              : combine_t<__nv_bfloat16>(tokens, top_k, rows, d, y, weight, row, out, st);
}

cudaError_t launch_combine_bwd(int tokens, int top_k, int rows, int d, bool fp32, const void* dout,
                               const void* y, const float* weight, const int* row, const int* pair,
                               const int* end, void* dy, float* dweight, cudaStream_t st) {
  if (tokens == 0 && rows == 0) return cudaSuccess;
  return fp32 ? combine_bwd_t<float>(tokens, top_k, rows, d, dout, y, weight, row, pair, end, dy,
                                     dweight, st)
              : combine_bwd_t<__nv_bfloat16>(tokens, top_k, rows, d, dout, y, weight, row, pair,
                                             end, dy, dweight, st);
}

cudaError_t launch_swiglu_fwd(int rows, int f, bool fp32, const void* gu, const int* end, void* ck,
                              cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  LaunchScope ls_("swiglu", st);
  const int grid = grid_for(((long long)rows * (ck_cols(f) / CK_GROUP) + 7) / 8, 152 * 8);
  if (fp32)
    swiglu_kernel<float><<<grid, 256, 0, st>>>(static_cast<const float*>(gu),
                                               static_cast<uint8_t*>(ck), end, rows, f);
  else
    swiglu_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(static_cast<const __nv_bfloat16*>(gu),
                                                       static_cast<uint8_t*>(ck), end, rows, f);
  return cudaGetLastError();
}

cudaError_t launch_swiglu_bwd(int rows, int f, bool fp32, const void* gu, const void* da,
                              const int* end, void* dgu, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  LaunchScope ls_("swiglu_bwd", st);
  const int grid = grid_for(((long long)rows * f + 255) / 256, 152 * 8);
  if (fp32)
    swiglu_bwd_kernel<float><<<grid, 256, 0, st>>>(
        static_cast<const float*>(gu), static_cast<const float*>(da), static_cast<float*>(dgu),
        end, rows, f);
  else
    swiglu_bwd_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(
        static_cast<const __nv_bfloat16*>(gu), static_cast<const __nv_bfloat16*>(da),
        static_cast<__nv_bfloat16*>(dgu), end, rows, f);
  return cudaGetLastError();
}

}  // namespace laga
