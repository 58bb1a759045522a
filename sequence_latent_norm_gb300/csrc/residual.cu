// The residual stream around a block (include/laga.h: laga_res_fwd,
// laga_res_bwd): x' = x + alpha s (N_post(y) gamma_post) and
// h = N_pre(x') gamma_pre, and their backward.
//
// With y^, x^ the normalised rows, r_y, r_x their 1/std, D = dL/dx' and
// [..] for LayerNorm only (means over the row's d channels):
//   e  = dh gamma_pre;       dx = D + r_x (e - [mean e] - x^ mean(e x^))
//   dz = alpha dx s;         f  = dz gamma_post
//   dy = r_y (f - [mean f] - y^ mean(f y^))            (no norm: dy = dz)
//   dgate = alpha dx s (1 - s) y^ gamma_post  (token gate: summed over d)
//   dalpha = sum dx s y^ gamma_post;  dgamma_post = sum_t dz y^;
//   dgamma_pre = sum_t dh x^
// Everything is fp32 between the loads and one rounding at the stores; dx
// enters the residual half before its rounding.
#include <float.h>

#include <algorithm>

#include "residual.cuh"

namespace laga {
namespace {

template <typename T>
LAGA_DEVINL float ld1(const void* p, long long i) { return to_f32(static_cast<const T*>(p)[i]); }
template <typename T>
LAGA_DEVINL void st1(void* p, long long i, float v) { static_cast<T*>(p)[i] = from_f32<T>(v); }

// ---------------------------------------------------- rows of any width
// (what the ring kernels do not take: widths that are no multiple of 8, and
// fp32 backwards too wide for a ring)
// One CTA per row, one element per access, the row's fp32 values in shared
// memory between the passes, and the backward's column sums beside them over
// all rows of a CTA.  Warp w owns the 128-channel groups w, w + GT / 32, ...,
// lane l the channels l, l + 32, l + 64, l + 96 of a group, in every pass, so
// a thread only ever reads what it wrote itself.
template <int GT, int K>
LAGA_DEVINL void block_sum(float (&v)[K], float* red) {   // red [GT / 32][K]
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = warp_sum(v[k]);
  __syncthreads();   // the previous reduction has been read
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) red[(threadIdx.x >> 5) * K + k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) {
    v[k] = 0.f;
    for (int w = 0; w < GT / 32; ++w) v[k] += red[w * K + k];
  }
}

template <int GT, typename F>
LAGA_DEVINL void for_cols(int d, F f) {
  for (int g = threadIdx.x >> 5; g * CK_GROUP < d; g += GT / 32)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = g * CK_GROUP + k * 32 + (threadIdx.x & 31);
      if (c < d) f(c);
    }
}

// A row's values v(c) as codes and scales
template <int GT, typename F>
LAGA_DEVINL void quantise_row(int d, uint8_t* row, F v) {
  const int cols = ck_cols(d), lane = threadIdx.x & 31;
  for (int g = threadIdx.x >> 5; g < cols / CK_GROUP; g += GT / 32) {
    float t[4], m = 0.f;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int c = g * CK_GROUP + k * 32 + lane;
      t[k] = c < d ? v(c) : 0.f;
      m = ck_max(m, t[k]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = ck_max(m, __shfl_xor_sync(0xffffffffu, m, o));
    float inv;
    const int s = ck_scale(m, &inv);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      row[g * CK_GROUP + k * 32 + lane] =
          s == CK_NAN ? 0 : (uint8_t)ck_code2(make_float2(t[k], 0.f), inv);
    if (lane == 0) row[cols + g] = (uint8_t)s;
  }
  for (int i = cols + cols / CK_GROUP + threadIdx.x; i < ck_pitch(d); i += GT) row[i] = 0;
}

// mean and 1/std of a row's values v(c)
template <int GT, typename F>
LAGA_DEVINL float2 row_stat(int d, float inv_d, int norm, float eps, float* red, F v) {
  if (norm == LAGA_NORM_NONE) return make_float2(0.f, 1.f);
  float mean = 0.f;
  if (norm == LAGA_NORM_LAYER) {
    float s[1] = {0.f};
    for_cols<GT>(d, [&](int c) { s[0] += v(c); });
    block_sum<GT, 1>(s, red);
    mean = s[0] * inv_d;
  }
  float q[1] = {0.f};
  for_cols<GT>(d, [&](int c) { const float t = v(c) - mean; q[0] += t * t; });
  block_sum<GT, 1>(q, red);
  return make_float2(mean, 1.f / sqrtf(q[0] * inv_d + eps));
}

template <typename T, int GT>
__global__ void __launch_bounds__(GT, 2048 / GT) res_fwd_rows_kernel(const ResArgs p) {
  extern __shared__ float xs[];   // [d]
  __shared__ float red[GT / 32];
  const int d = p.d, pitch = ck_pitch(d);
  for (long long r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const long long o = r * d;
    for_cols<GT>(d, [&](int c) { xs[c] = ld1<T>(p.x.x, o + c); });
    if (p.post) {
      const float alpha = *p.x.alpha;
      const float2 st = row_stat<GT>(d, p.inv_d, p.norm_post, p.eps, red,
                                 [&](int c) { return ld1<T>(p.x.y, o + c); });
      auto hat = [&](int c) { return (ld1<T>(p.x.y, o + c) - st.x) * st.y; };
      for_cols<GT>(d, [&](int c) {
        float z = hat(c);
        if (p.norm_post != LAGA_NORM_NONE) z *= p.x.gamma_post[c];
        if (p.gate != LAGA_GATE_NONE)
          z *= sigmoid_pair(ld1<T>(p.x.gate, p.gate == LAGA_GATE_FULL ? o + c : r)).x;
        xs[c] += alpha * z;
        st1<T>(p.x.x_out, o + c, xs[c]);
      });
      if (p.ckpt) quantise_row<GT>(d, static_cast<uint8_t*>(p.x.ck_y) + r * pitch, hat);
      if (threadIdx.x == 0) reinterpret_cast<float2*>(p.x.stat_post)[r] = st;
    }
    if (p.pre) {
      const float2 st = row_stat<GT>(d, p.inv_d, p.norm_pre, p.eps, red, [&](int c) { return xs[c]; });
      auto hat = [&](int c) { return (xs[c] - st.x) * st.y; };
      for_cols<GT>(d, [&](int c) { st1<T>(p.x.h, o + c, hat(c) * p.x.gamma_pre[c]); });
      if (p.ckpt) quantise_row<GT>(d, static_cast<uint8_t*>(p.x.ck_x) + r * pitch, hat);
      if (threadIdx.x == 0) reinterpret_cast<float2*>(p.x.stat_pre)[r] = st;
    }
  }
}

// Normalised element c of row r: from its checkpoint, or from the kept tensor
template <typename T>
LAGA_DEVINL float kept_hat(const void* kept, int ckpt, int d, long long r, int c, float2 st) {
  if (!ckpt) return (ld1<T>(kept, r * d + c) - st.x) * st.y;
  const uint8_t* row = static_cast<const uint8_t*>(kept) + r * ck_pitch(d);
  return ck_value2(row[c], ck_unit(row[ck_cols(d) + c / CK_GROUP])).x;
}

template <typename T, int GT>
__global__ void __launch_bounds__(GT, 2048 / GT) res_bwd_rows_kernel(const ResArgs p) {
  extern __shared__ float ds[];   // [3][d]: dx, then f; the column sums
  __shared__ float red[4 * GT / 32];
  const int d = p.d;
  float d_alpha = 0.f;
  float *const pp = ds + d, *const pq = ds + 2 * d;
  for_cols<GT>(d, [&](int c) { pp[c] = pq[c] = 0.f; });
  for (long long r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const long long o = r * d;
    if (p.pre) {
      const float2 st = reinterpret_cast<const float2*>(p.x.stat_pre)[r];
      auto hat = [&](int c) { return kept_hat<T>(p.x.kept_x, p.ckpt, d, r, c, st); };
      float s[2] = {0.f, 0.f};
      for_cols<GT>(d, [&](int c) {
        const float dh = ld1<T>(p.x.dh, o + c), x = hat(c), e = dh * p.x.gamma_pre[c];
        pq[c] += dh * x;
        s[0] += e;
        s[1] += e * x;
      });
      block_sum<GT, 2>(s, red);
      const float m0 = p.norm_pre == LAGA_NORM_LAYER ? s[0] * p.inv_d : 0.f, m1 = s[1] * p.inv_d;
      for_cols<GT>(d, [&](int c) {
        const float e = ld1<T>(p.x.dh, o + c) * p.x.gamma_pre[c];
        const float D = p.x.dx_out ? ld1<T>(p.x.dx_out, o + c) : 0.f;
        ds[c] = D + st.y * (e - m0 - hat(c) * m1);
        st1<T>(p.x.dx, o + c, ds[c]);
      });
    } else {
      for_cols<GT>(d, [&](int c) { ds[c] = ld1<T>(p.x.dx_out, o + c); });
    }
    if (p.post) {
      const float alpha = *p.x.alpha;
      const float2 st = reinterpret_cast<const float2*>(p.x.stat_post)[r];
      float s[4] = {0.f, 0.f, 0.f, 0.f};   // f, f y^, dx s z, token gate
      for_cols<GT>(d, [&](int c) {
        const float y = kept_hat<T>(p.x.kept_y, p.ckpt, d, r, c, st);
        const float g = p.norm_post != LAGA_NORM_NONE ? p.x.gamma_post[c] : 1.f;
        float2 sg = make_float2(1.f, 0.f);
        if (p.gate != LAGA_GATE_NONE)
          sg = sigmoid_pair(ld1<T>(p.x.gate, p.gate == LAGA_GATE_FULL ? o + c : r));
        const float ad = alpha * ds[c], z = y * g, dz = ad * sg.x, f = dz * g;
        s[2] += ds[c] * sg.x * z;
        const float da = dz * sg.y * z;
        if (p.gate == LAGA_GATE_FULL) st1<T>(p.x.dgate, o + c, da);
        s[3] += da;
        if (p.norm_post != LAGA_NORM_NONE) pp[c] += dz * y;
        s[0] += f;
        s[1] += f * y;
        ds[c] = f;
      });
      block_sum<GT, 4>(s, red);
      d_alpha += s[2];
      if (p.gate == LAGA_GATE_TOKEN && threadIdx.x == 0) st1<T>(p.x.dgate, r, s[3]);
      const bool none = p.norm_post == LAGA_NORM_NONE;
      const float m0 = p.norm_post == LAGA_NORM_LAYER ? s[0] * p.inv_d : 0.f;
      const float m1 = none ? 0.f : s[1] * p.inv_d;
      for_cols<GT>(d, [&](int c) {
        const float y = none ? 0.f : kept_hat<T>(p.x.kept_y, p.ckpt, d, r, c, st);
        st1<T>(p.x.dy, o + c, (none ? 1.f : st.y) * (ds[c] - m0 - y * m1));
      });
    }
  }
  const long long slot = (long long)blockIdx.x * d;
  for_cols<GT>(d, [&](int c) {
    if (p.post && p.norm_post != LAGA_NORM_NONE) p.part_post[slot + c] = pp[c];
    if (p.pre) p.part_pre[slot + c] = pq[c];
  });
  if (p.post && threadIdx.x == 0) p.part_alpha[blockIdx.x] = d_alpha;
}

// Sums of the column partials over their slots, CW columns a block: 1024 / CW
// chains of every so many'th slot, four loads at a time, added up in order.  32
// columns, or, up to 1024 channels, 8 (one 32-byte sector of a slot), so that
// there are blocks enough: 512 channels 8 us with 8 and 15 us with 32 columns,
// 7168 channels 15 us and 9 us.  blockIdx.y 0: gamma_post, 1: gamma_pre; block
// (0, 2): alpha.
template <int CW>
__global__ void __launch_bounds__(1024) res_colsum_kernel(const float* part_post, const float* part_pre,
                                                          const float* part_alpha, int slots, int d,
                                                          float* dg_post, float* dg_pre,
                                                          float* dalpha) {
  constexpr int NG = 1024 / CW;
  __shared__ float sm[NG][CW + 1], sm2[8][CW + 1];
  const int tid = threadIdx.x, col = tid % CW, g = tid / CW;
  if (blockIdx.y == 2) {
    if (blockIdx.x || tid >= 32 || !dalpha) return;
    float s = 0.f;
    for (int k = tid; k < slots; k += 32) s += part_alpha[k];
    s = warp_sum(s);
    if (tid == 0) *dalpha = s;
    return;
  }
  const float* part = blockIdx.y ? part_pre : part_post;
  float* out = blockIdx.y ? dg_pre : dg_post;
  if (!out) return;
  const int c = blockIdx.x * CW + col;
  float s = 0.f;
  if (c < d)
    for (int k0 = g; k0 < slots; k0 += NG * 4) {
      float v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = k0 + NG * i;
        v[i] = k < slots ? part[(long long)k * d + c] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) s += v[i];
    }
  sm[g][col] = s;
  __syncthreads();
  if (g < 8) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < NG / 8; ++i) s += sm[g * (NG / 8) + i][col];
    sm2[g][col] = s;
  }
  __syncthreads();
  if (g == 0 && c < d) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) s += sm2[i][col];
    out[c] = s;
  }
}

size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Rows of any width: 2048 threads an SM (32 registers each), which hide the
// latency of the scalar accesses, in CTAs of 256 threads, or of 1024 where
// shared memory does not hold `arrays` fp32 rows for eight CTAs.  With 41
// registers and so fewer threads the forward took 110 us instead of 87 (4096 x
// 5001 bf16), and with 256 threads throughout, the sums in global memory, the
// backward 443 us instead of 297.
bool rows_wide(int d, int arrays) { return arrays * d * 4 + 2048 > 220 * 1024 / 8; }
int rows_ctas(int d, int arrays) {
  return std::max(1, std::min(rows_wide(d, arrays) ? 2 : 8, 220 * 1024 / (arrays * d * 4 + 2048)));
}

// Column partial slots of a backward launch
int bwd_slots(const laga_res_dims& d) {
  return ring_ok(d, true) ? ring_slots(d) : std::min(d.rows, kSms * rows_ctas(d.d, 3));
}

ResArgs make_args(const laga_res_dims& d, const ResPtrs& x) {
  ResArgs a{};
  a.rows = d.rows; a.d = d.d;
  a.post = d.post; a.pre = d.pre;
  a.norm_post = d.norm_post; a.norm_pre = d.norm_pre;
  a.gate = d.post ? d.gate : LAGA_GATE_NONE;
  a.ckpt = d.ckpt;
  a.eps = d.eps;
  a.inv_d = 1.f / (float)d.d;
  a.x = x;
  return a;
}

// Lets the scalar kernel f have `arrays` fp32 rows of the widest width, whatever
// this call needs: the limit belongs to the kernel, and another thread may be
// about to launch it for another width.
template <typename F>
cudaError_t allow_rows(F* f, int arrays) {
  return cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, arrays * CK_MAX_D * 4);
}

}  // namespace

laga_status res_check(const laga_res_dims* p) {
  if (!p) return LAGA_ERR_ARG;
  const laga_res_dims& d = *p;
  if (d.rows < 0 || d.d < 1 || d.d > CK_MAX_D) return LAGA_ERR_ARG;
  if ((d.post != 0 && d.post != 1) || (d.pre != 0 && d.pre != 1) || !(d.post || d.pre))
    return LAGA_ERR_ARG;
  if (d.ckpt != 0 && d.ckpt != 1) return LAGA_ERR_ARG;
  if (!(d.eps > 0.f) || !(d.eps <= FLT_MAX)) return LAGA_ERR_ARG;
  if (d.norm_post != LAGA_NORM_LAYER && d.norm_post != LAGA_NORM_RMS &&
      d.norm_post != LAGA_NORM_NONE)
    return LAGA_ERR_ARG;
  if (d.norm_pre != LAGA_NORM_LAYER && d.norm_pre != LAGA_NORM_RMS) return LAGA_ERR_ARG;
  if (d.gate != LAGA_GATE_NONE && d.gate != LAGA_GATE_TOKEN && d.gate != LAGA_GATE_FULL)
    return LAGA_ERR_ARG;
  if (d.io_dtype != LAGA_BF16 && d.io_dtype != LAGA_FP32) return LAGA_ERR_ARG;
  return LAGA_OK;
}

size_t res_ws_bytes(const laga_res_dims& d) {
  const size_t slots = (size_t)bwd_slots(d);
  return 2 * up256(slots * d.d * 4) + up256(slots * 4);
}

cudaError_t launch_res_fwd(const laga_res_dims& d, const ResPtrs& x, cudaStream_t st) {
  if (d.rows == 0) return cudaSuccess;
  const ResArgs a = make_args(d, x);
  if (ring_ok(d, false)) return launch_ring_fwd(d, a, st);
  const size_t smem = (size_t)d.d * 4;
  const bool f32 = d.io_dtype == LAGA_FP32, wide = rows_wide(d.d, 1);
  auto k = wide ? (f32 ? res_fwd_rows_kernel<float, 1024> : res_fwd_rows_kernel<__nv_bfloat16, 1024>)
                : (f32 ? res_fwd_rows_kernel<float, 256> : res_fwd_rows_kernel<__nv_bfloat16, 256>);
  cudaError_t e = allow_rows(k, 1);
  if (e != cudaSuccess) return e;
  LaunchScope ls_("res_fwd", st);
  k<<<std::min(d.rows, kSms * rows_ctas(d.d, 1)), wide ? 1024 : 256, smem, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_res_bwd(const laga_res_dims& d, const ResPtrs& x, cudaStream_t st) {
  ResArgs a = make_args(d, x);
  const int slots = bwd_slots(d);
  a.part_post = reinterpret_cast<float*>(x.ws);
  a.part_pre = reinterpret_cast<float*>(x.ws + up256((size_t)slots * d.d * 4));
  a.part_alpha = reinterpret_cast<float*>(x.ws + 2 * up256((size_t)slots * d.d * 4));
  cudaError_t e;
  if (d.rows > 0 && ring_ok(d, true)) {
    if ((e = launch_ring_bwd(d, a, st)) != cudaSuccess) return e;
  } else if (d.rows > 0) {
    const size_t smem = (size_t)3 * d.d * 4;
    const bool f32 = d.io_dtype == LAGA_FP32, wide = rows_wide(d.d, 3);
    auto k = wide
                 ? (f32 ? res_bwd_rows_kernel<float, 1024> : res_bwd_rows_kernel<__nv_bfloat16, 1024>)
                 : (f32 ? res_bwd_rows_kernel<float, 256> : res_bwd_rows_kernel<__nv_bfloat16, 256>);
    if ((e = allow_rows(k, 3)) != cudaSuccess) return e;
    LaunchScope ls_("res_bwd", st);
    k<<<slots, wide ? 1024 : 256, smem, st>>>(a);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  LaunchScope ls_("res_colsum", st);
  const int cw = d.d <= 1024 ? 8 : 32;
  const auto k = cw == 8 ? res_colsum_kernel<8> : res_colsum_kernel<32>;
  k<<<dim3((d.d + cw - 1) / cw, 3), 1024, 0, st>>>(
      a.part_post, a.part_pre, a.part_alpha, slots, d.d,
      d.post && d.norm_post != LAGA_NORM_NONE ? x.dgamma_post : nullptr,
      d.pre ? x.dgamma_pre : nullptr, d.post ? x.dalpha : nullptr);
  return cudaGetLastError();
}

}  // namespace laga
