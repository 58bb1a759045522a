// Rows to experts and back, and the experts' gated activation (include/laga.h:
// laga_spread8, laga_combine_*, laga_swiglu_*).  What moves rows is bound by HBM, the
// activation by HBM and its instructions.
#include <algorithm>

#include "ckpt8.cuh"
#include "common.cuh"
#include "kernels.h"
#include "ops.h"
#include "vec8.cuh"

namespace laga {
namespace {

// ------------------------------------------------------------------ rows
// A warp copies one row of codes, 16 bytes a lane and eight such loads at a
// time (16384 rows of 7232 bytes from 2048: 27 us, 35 us one at a time).
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
    for (int v0 = lane; v0 < vecs; v0 += 32 * 8) {
      uint4 q[8];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (v0 + 32 * k < vecs) q[k] = src[v0 + 32 * k];
#pragma unroll
      for (int k = 0; k < 8; ++k)
        if (v0 + 32 * k < vecs) dst[v0 + 32 * k] = q[k];
    }
  }
}

// out_t = sum_j w_tj y[row_tj]: a thread V channels of a token.  A choice that a
// NaN left without an expert makes it a NaN, also under weights of 1.
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
      if (r < 0 || r >= rows) {
        if (r == ROUTE_ROW_NAN)
#pragma unroll
          for (int k = 0; k < (V + 1) / 2; ++k)
            acc[k].x = acc[k].y = __int_as_float(0x7fc00000);
        continue;
      }
      const float w = weight ? weight[t * top_k + j] : 1.f;
      float2 f[(V + 1) / 2];
      load_vec<V>(y + (long long)r * d + c, f);
#pragma unroll
      for (int k = 0; k < (V + 1) / 2; ++k) acc[k] = __ffma2_rn(f[k], make_float2(w, w), acc[k]);
    }
    store_vec<V>(out + t * d + c, acc);
  }
}

// dy[r] = w dout_t, dw = <dout_t, y[r]> of the row's pair: a warp a row, with
// LOADS vectors of each side under way.  It goes by rows, not by pairs: y and dy
// stream through HBM in order then, and dout, which every choice reads, stays in
// L2.  (16384 x 7168 rows of 2048 tokens: 91 us, by pairs 131 to 183 us.)  Rows of no
// pair get zeros, pairs without a row a dw of zero.
constexpr int LOADS = 4;

// What a row has to do with its pair.
struct PairOf {
  bool on;
  int q;
  long long token;
  float w;
  LAGA_DEVINL PairOf(const int* pair, const float* weight, long long r, long long pairs,
                     int top_k) {
    q = pair[r];
    on = q >= 0 && q < pairs;
    token = on ? q / top_k : 0;
    w = on ? weight ? weight[q] : 1.f : 0.f;
  }
};

// The pairs without a row.
LAGA_DEVINL void zero_dweight(float* dweight, const int* row, long long pairs, int rows) {
  for (long long q = blockIdx.x * 256LL + threadIdx.x; q < pairs; q += gridDim.x * 256LL)
    if (row[q] < 0 || row[q] >= rows) dweight[q] = 0.f;
}

template <typename T>
__global__ void __launch_bounds__(256, 4)
    combine_bwd_kernel(const T* __restrict__ dout, const T* __restrict__ y,
                       const float* __restrict__ weight, const int* __restrict__ row,
                       const int* __restrict__ pair, const int* __restrict__ end,
                       T* __restrict__ dy, float* __restrict__ dweight, int tokens, int top_k,
                       int rows, int d) {
  constexpr int V = vec16<T>, P = V / 2;
  const int vecs = d / V, lane = threadIdx.x & 31;
  const long long pairs = (long long)tokens * top_k;
  const int n = rows > 0 ? min(rows, *end) : 0;
  for (long long r = blockIdx.x * 8LL + (threadIdx.x >> 5); r < n; r += gridDim.x * 8LL) {
    const PairOf o(pair, weight, r, pairs, top_k);
    const uint4* src = reinterpret_cast<const uint4*>(dout + o.token * d);
    const uint4* old = reinterpret_cast<const uint4*>(y + r * d);
    uint4* dst = reinterpret_cast<uint4*>(dy + r * d);
    float2 dot = make_float2(0.f, 0.f);
    for (int v0 = lane; v0 < vecs; v0 += 32 * LOADS) {
      uint4 g[LOADS], f[LOADS];
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        const int v = v0 + 32 * i;
        g[i] = f[i] = make_uint4(0, 0, 0, 0);
        if (o.on && v < vecs) {
          g[i] = __ldg(src + v);
          if (dweight) f[i] = __ldcs(old + v);
        }
      }
#pragma unroll
      for (int i = 0; i < LOADS; ++i) {
        float2 a[P], b[P];
        open16(g[i], dout, a);
        open16(f[i], dout, b);
#pragma unroll
        for (int k = 0; k < P; ++k) {
          dot = __ffma2_rn(a[k], b[k], dot);
          a[k] = __fmul2_rn(a[k], make_float2(o.w, o.w));
        }
        if (v0 + 32 * i < vecs) dst[v0 + 32 * i] = close16(dout, a);
      }
    }
    if (!dweight || !o.on) continue;
    const float sum = warp_sum(dot.x + dot.y);
    if (lane == 0) dweight[o.q] = sum;
  }
  if (dweight) zero_dweight(dweight, row, pairs, rows);
}

// Other widths, channel by channel.
template <typename T>
__global__ void __launch_bounds__(256)
    combine_bwd1_kernel(const T* __restrict__ dout, const T* __restrict__ y,
                        const float* __restrict__ weight, const int* __restrict__ row,
                        const int* __restrict__ pair, const int* __restrict__ end,
                        T* __restrict__ dy, float* __restrict__ dweight, int tokens, int top_k,
                        int rows, int d) {
  const int lane = threadIdx.x & 31;
  const long long pairs = (long long)tokens * top_k;
  const int n = rows > 0 ? min(rows, *end) : 0;
  for (long long r = blockIdx.x * 8LL + (threadIdx.x >> 5); r < n; r += gridDim.x * 8LL) {
    const PairOf o(pair, weight, r, pairs, top_k);
    float dot = 0.f;
#pragma unroll 4
    for (int c = lane; c < d; c += 32) {
      const float g = o.on ? to_f32(dout[o.token * d + c]) : 0.f;
      if (o.on && dweight) dot = fmaf(g, to_f32(y[r * d + c]), dot);
      dy[r * d + c] = from_f32<T>(g * o.w);
    }
    if (!dweight || !o.on) continue;
    dot = warp_sum(dot);
    if (lane == 0) dweight[o.q] = dot;
  }
  if (dweight) zero_dweight(dweight, row, pairs, rows);
}

// ------------------------------------------------------------------ activation
// Each kernel moves 4 to 10 bytes a channel and has some 25 instructions for it
// at that rate, so the sigmoid is two special functions; channels come in
// vectors of 8 where the width allows.  (16384 x 2048 bf16: 34 us forward, and 82 us
// with expf, a division and single channels.)

// sigmoid(g) and 1 - sigmoid(g) = e^-g sigmoid(g), each within 6 units of its
// last place: the exponent's product with log2 e is carried in two parts, since
// what it loses moves codes across their borders.  Below -87.3 the sigmoid
// would be subnormal: both are zero.  Above 104 e^-g is zero, and g stops there:
// from 2.4e38 on the product would be infinite and its second part no number.
constexpr float C = -1.44269502f, C_LO = -1.92596303e-8f, LN2 = 0.693147182f;
LAGA_DEVINL float2 sigmoid2(float g) {
  float e, s;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(g) : "f"(g), "f"(-88.5f));
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(g) : "f"(g), "f"(104.f));
  const float t = g * C;
  const float lo = fmaf(g, C_LO, fmaf(g, C, -t));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  e = fmaf(e, lo * LN2, e);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
  return make_float2(s, e * s);
}
// sigmoid(g) alone, the same bits, for which e^-g may be infinite: there the
// second part, which has no use, is left out.  (A test instead of two bounds: 16384
// x 2048 bf16 takes 33.8 us, 35.6 us with sigmoid2.)
LAGA_DEVINL float sigmoid(float g) {
  float e, s;
  const float t = g * C;
  const float lo = fmaf(g, C_LO, fmaf(g, C, -t));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(t));
  if (fabsf(g) < 88.5f) e = fmaf(e, lo * LN2, e);
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
  return s;
}

// Codes of a group's values, `lanes` neighbouring lanes of V each.
template <int V>
LAGA_DEVINL float group_max(const float (&t)[V]) {
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < V; ++k) m = ck_max(m, t[k]);
#pragma unroll
  for (int o = CK_GROUP / V / 2; o > 0; o >>= 1) m = ck_max(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// a = silu(g) u.  A thread V channels, CK_GROUP / V neighbouring threads a
// group; widths that are no multiple of 8 go 4 channels at a time, one by one.
template <typename T, int V>
__global__ void __launch_bounds__(256)
    swiglu_kernel(const T* __restrict__ gu, uint8_t* __restrict__ ck, const int* __restrict__ end,
                  int rows, int f) {
  const int cols = ck_cols(f), vpr = cols / V, pitch = ck_pitch(f);
  const int pad = pitch - cols - cols / CK_GROUP;
  const int n_rows = end ? min(rows, *end) : rows;
  for (long long r0 = (long long)blockIdx.x * 2; r0 < n_rows; r0 += (long long)gridDim.x * 2) {
    const int n = (int)min(2LL, n_rows - r0) * vpr;
    // whole warps go round, so that every lane of a group is there
    for (int i0 = threadIdx.x & ~31; i0 < n; i0 += 256) {
      const int i = i0 + (threadIdx.x & 31);
      const int r = i / vpr, v = i - r * vpr;
      const T* src = gu + (r0 + r) * 2 * f + v * V;
      float t[V];
      if constexpr (V == 8) {
        float2 g[4] = {}, u[4] = {};
        if (i < n && v * 8 < f) {
          load_vec<8>(src, g);
          load_vec<8>(src + f, u);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          t[2 * k] = g[k].x * sigmoid(g[k].x) * u[k].x;
          t[2 * k + 1] = g[k].y * sigmoid(g[k].y) * u[k].y;
        }
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) {
          t[k] = 0.f;
          if (i < n && v * V + k < f) {
            const float g = to_f32(src[k]);
            t[k] = g * sigmoid(g) * to_f32(src[f + k]);
          }
        }
      }
      float inv;
      const int s = ck_scale(group_max<V>(t), &inv);
      if (i >= n) continue;
      uint8_t* row = ck + (r0 + r) * pitch;
      uint32_t q[V / 4];
#pragma unroll
      for (int k = 0; k < V / 4; ++k) {
        q[k] = ck_code2(make_float2(t[4 * k], t[4 * k + 1]), inv) |
               ck_code2(make_float2(t[4 * k + 2], t[4 * k + 3]), inv) << 16;
        if (s == CK_NAN) q[k] = 0u;
      }
      if constexpr (V == 8)
        reinterpret_cast<uint2*>(row)[v] = make_uint2(q[0], q[1]);
      else
        reinterpret_cast<uint32_t*>(row)[v] = q[0];
      if (v % (CK_GROUP / V) == 0) row[cols + v / (CK_GROUP / V)] = (uint8_t)s;
      if (v < pad) row[cols + cols / CK_GROUP + v] = 0;
    }
  }
}

// dg = da u sigma (1 + g (1 - sigma)), du = da g sigma: a thread V channels.
template <typename T, int V>
__global__ void __launch_bounds__(256)
    swiglu_bwd_kernel(const T* __restrict__ gu, const T* __restrict__ da, T* __restrict__ dgu,
                      const int* __restrict__ end, int rows, int f) {
  constexpr int P = (V + 1) / 2;
  const int vpr = f / V;
  const long long n = (long long)(end ? min(rows, *end) : rows) * vpr;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < n; i += gridDim.x * 256LL) {
    const long long r = i / vpr;
    const int c = (int)(i - r * vpr) * V;
    const long long o = r * 2 * f + c;
    float2 g[P], u[P], d[P];
    load_vec<V>(gu + o, g);
    load_vec<V>(gu + o + f, u);
    load_vec<V>(da + r * f + c, d);
#pragma unroll
    for (int k = 0; k < P; ++k) {
      const float2 sx = sigmoid2(g[k].x), sy = sigmoid2(g[k].y);
      const float2 ds = __fmul2_rn(d[k], make_float2(sx.x, sy.x));
      u[k] = __fmul2_rn(ds, u[k]);
      u[k].x *= fmaf(g[k].x, sx.y, 1.f);
      u[k].y *= fmaf(g[k].y, sy.y, 1.f);
      g[k] = __fmul2_rn(ds, g[k]);
    }
    store_vec<V>(dgu + o, u);
    store_vec<V>(dgu + o + f, g);
  }
}

int grid_for(long long blocks, int most) {
  return (int)std::max<long long>(1, std::min<long long>(blocks, most));
}

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
  const long long by_row = ((long long)rows + 7) / 8;
  const int grid = grid_for(std::max(by_row, ((long long)tokens * top_k + 255) / 256), 152 * 32);
  const T *g = static_cast<const T*>(dout), *f = static_cast<const T*>(y);
  auto k = d % vec16<T> == 0 ? combine_bwd_kernel<T> : combine_bwd1_kernel<T>;
  k<<<grid, 256, 0, st>>>(g, f, weight, row, pair, end, static_cast<T*>(dy), dweight, tokens,
                          top_k, rows, d);
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

namespace {
template <typename T>
void swiglu_t(int rows, int f, const void* gu, const int* end, void* ck, cudaStream_t st) {
  // more blocks than fit, to even out the end (16384 x 2048: 36 us with a wave)
  const int grid = grid_for(((long long)rows + 1) / 2, 152 * 32);
  auto k = f % 8 == 0 ? swiglu_kernel<T, 8> : swiglu_kernel<T, 4>;
  k<<<grid, 256, 0, st>>>(static_cast<const T*>(gu), static_cast<uint8_t*>(ck), end, rows, f);
}
template <typename T>
void swiglu_bwd_t(int rows, int f, const void* gu, const void* da, const int* end, void* dgu,
                  cudaStream_t st) {
  const int v = f % 8 == 0 ? 8 : 1;
  const int grid = grid_for(((long long)rows * (f / v) + 255) / 256, 152 * 8);
  auto k = v == 8 ? swiglu_bwd_kernel<T, 8> : swiglu_bwd_kernel<T, 1>;
  k<<<grid, 256, 0, st>>>(static_cast<const T*>(gu), static_cast<const T*>(da),
                          static_cast<T*>(dgu), end, rows, f);
}
}  // namespace

cudaError_t launch_swiglu_fwd(int rows, int f, bool fp32, const void* gu, const int* end, void* ck,
                              cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  LaunchScope ls_("swiglu", st);
  if (fp32)
    swiglu_t<float>(rows, f, gu, end, ck, st);
  else
    swiglu_t<__nv_bfloat16>(rows, f, gu, end, ck, st);
  return cudaGetLastError();
}

cudaError_t launch_swiglu_bwd(int rows, int f, bool fp32, const void* gu, const void* da,
                              const int* end, void* dgu, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  LaunchScope ls_("swiglu_bwd", st);
  if (fp32)
    swiglu_bwd_t<float>(rows, f, gu, da, end, dgu, st);
  else
    swiglu_bwd_t<__nv_bfloat16>(rows, f, gu, da, end, dgu, st);
  return cudaGetLastError();
}

}  // namespace laga
