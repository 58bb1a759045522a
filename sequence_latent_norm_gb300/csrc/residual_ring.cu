// The residual stream for rows of a multiple of 8 channels (the formulas are
// in residual.cu).  All of it is bound by HBM: per element a bf16 junction
// with a full gate moves 10 bytes forward and, from 8-bit checkpoints, 12
// backward, against ~30 and ~60 arithmetic instructions.
//
// A CTA of 512 threads per SM is cut into teams; a team walks rows, one at a
// time, and each team has a ring of row buffers in shared memory that one
// thread keeps filled with bulk copies (cp.async.bulk, one per input tensor
// and row, completion counted on the buffer's mbarrier).  So the loads of the
// next rows are in flight while a row is worked on, whatever the reductions
// in the middle of a row wait for.  Inside a row a thread owns the 8-channel
// vectors tl, tl + TEAM, ...: 16 neighbouring threads hold one checkpoint
// group.  The gains sit in shared memory for the whole launch.  Column sums
// (the gains' gradients) stay in registers over all of a team's rows and are
// written once, as one partial row per team; residual.cu adds those up.
#include <algorithm>

#include "residual.cuh"
#include "sm100.cuh"

namespace laga {
namespace {
using namespace sm100;

constexpr int THREADS = 512;
constexpr int MAX_DEPTH = 4;
constexpr int SMEM_MAX = 225 * 1024;

struct Src {
  const uint8_t* base;
  uint32_t row_bytes, off;          // bytes of a row, and its place in a row buffer
};
struct RingArgs {
  Src src[5];
  int depth;
  uint32_t stage_bytes, gain_bytes;  // gain_bytes 0: the gains are read from global memory
};
enum FwdSrc { F_X, F_Y, F_G };
enum BwdSrc { B_D, B_DH, B_X, B_Y, B_G };

// Bulk copy global -> shared, 16-byte aligned addresses and size.
LAGA_DEVINL void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
          smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// 8 consecutive elements
template <typename T>
struct Vec;
template <>
struct Vec<__nv_bfloat16> {
  static LAGA_DEVINL void load(const uint8_t* p, int v, float (&f)[8]) {
    const uint4 w = reinterpret_cast<const uint4*>(p)[v];
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      f[2 * k] = __uint_as_float(u[k] << 16);
      f[2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
    }
  }
  static LAGA_DEVINL void store(void* p, long long v, const float (&f)[8]) {
    reinterpret_cast<uint4*>(p)[v] = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                                pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
  }
};
template <>
struct Vec<float> {
  static LAGA_DEVINL void load(const uint8_t* p, int v, float (&f)[8]) {
    const float4 a = reinterpret_cast<const float4*>(p)[2 * v];
    const float4 b = reinterpret_cast<const float4*>(p)[2 * v + 1];
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
  static LAGA_DEVINL void store(void* p, long long v, const float (&f)[8]) {
    reinterpret_cast<float4*>(p)[2 * v] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[2 * v + 1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};

// A row's gain: in shared memory as two planes of four floats per vector, so
// that 16-byte accesses of neighbouring threads do not collide, or global.
struct Gain {
  const float *sm, *g;
  int nvec;
  LAGA_DEVINL void load(int v, float (&f)[8]) const {
    const float4 a = sm ? reinterpret_cast<const float4*>(sm)[v]
                        : __ldg(reinterpret_cast<const float4*>(g) + 2 * v);
    const float4 b = sm ? reinterpret_cast<const float4*>(sm)[nvec + v]
                        : __ldg(reinterpret_cast<const float4*>(g) + 2 * v + 1);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};

LAGA_DEVINL void copy_gain(float* dst, const float* src, int d) {
  for (int c = threadIdx.x; c < d; c += THREADS)
    dst[((c >> 2) & 1) * (d >> 1) + (c >> 3) * 4 + (c & 3)] = src[c];
}

template <int TEAM>
LAGA_DEVINL void team_sync(int team) {
  if (TEAM == 32)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(1 + team), "n"(TEAM) : "memory");
}

// Sum K values over a team.  Two alternating slots of partial sums: a slot is
// written again two reductions later, behind the barrier in between.
template <int TEAM, int K>
LAGA_DEVINL void team_sum(float (&v)[K], float (*red)[THREADS / 32][4], int team, int& slot) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = warp_sum(v[k]);
  if (TEAM == 32) return;
  constexpr int NW = TEAM / 32;
  const int w = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int k = 0; k < K; ++k) red[slot][w][k] = v[k];
  team_sync<TEAM>(team);
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = 0.f;
#pragma unroll
  for (int i = 0; i < NW; ++i)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += red[slot][team * NW + i][k];
  slot ^= 1;
}

// One vector of normalised values as codes, with its group's scale (16
// neighbouring lanes hold the group; every lane of the warp takes part).
LAGA_DEVINL void quantise8(uint8_t* row, int v, int cols, const float (&f)[8]) {
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = fmaxf(m, ck_mag(f[k]));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  float inv;
  const int s = ck_scale(m, &inv);
  if (v * 8 < cols) {
    reinterpret_cast<uint2*>(row)[v] =
        make_uint2(ck_code2(f[0], f[1], inv) | ck_code2(f[2], f[3], inv) << 16,
                   ck_code2(f[4], f[5], inv) | ck_code2(f[6], f[7], inv) << 16);
    if ((v & 15) == 0) row[cols + (v >> 4)] = (uint8_t)s;
  }
}

// One vector of a kept row: the checkpoint's values, or (kept - mean) / std.
template <typename T>
LAGA_DEVINL void kept8(const uint8_t* row, int ckpt, int cols, int v, float2 st, float (&f)[8]) {
  if (ckpt) {
    const uint2 q = reinterpret_cast<const uint2*>(row)[v];
    const float unit = ck_unit(row[cols + (v >> 4)]);
    const uint32_t c[4] = {q.x & 0xffffu, q.x >> 16, q.y & 0xffffu, q.y >> 16};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 t = ck_value2(c[k], unit);
      f[2 * k] = t.x;
      f[2 * k + 1] = t.y;
    }
  } else {
    Vec<T>::load(row, v, f);
#pragma unroll
    for (int k = 0; k < 8; ++k) f[k] = (f[k] - st.x) * st.y;
  }
}

// What both directions set up: barriers, gains, and a team's place.
template <int TEAM>
struct Ring {
  uint64_t* bar;        // this team's barriers
  uint8_t* buf;         // this team's row buffers
  int team, tl, depth;
  uint32_t stage_bytes;

  LAGA_DEVINL void issue(const RingArgs& q, int st, long long row) const {
    mbar_arrive_expect_tx(&bar[st], q.stage_bytes);
    for (int i = 0; i < 5; ++i)
      if (q.src[i].row_bytes)
        bulk_load(buf + st * stage_bytes + q.src[i].off, q.src[i].base + row * q.src[i].row_bytes,
                  q.src[i].row_bytes, &bar[st]);
  }
};

extern __shared__ __align__(128) uint8_t dyn_smem[];

template <int TEAM>
LAGA_DEVINL Ring<TEAM> ring_setup(const ResArgs& p, const RingArgs& q, uint64_t (*bars)[MAX_DEPTH],
                                  Gain& g_post, Gain& g_pre) {
  constexpr int TEAMS = THREADS / TEAM;
  Ring<TEAM> r;
  r.team = threadIdx.x / TEAM;
  r.tl = threadIdx.x % TEAM;
  r.depth = q.depth;
  r.stage_bytes = q.stage_bytes;
  r.bar = bars[r.team];
  r.buf = dyn_smem + q.gain_bytes + (size_t)r.team * q.depth * q.stage_bytes;
  if (threadIdx.x == 0) {
    for (int t = 0; t < TEAMS; ++t)
      for (int s = 0; s < q.depth; ++s) mbar_init(&bars[t][s], 1);
    fence_barrier_init();
  }
  const bool gain = p.post && p.norm_post != LAGA_NORM_NONE;
  float* sg = reinterpret_cast<float*>(dyn_smem);
  g_post = {nullptr, p.x.gamma_post, p.d >> 3};
  g_pre = {nullptr, p.x.gamma_pre, p.d >> 3};
  if (q.gain_bytes) {
    if (gain) {
      copy_gain(sg, p.x.gamma_post, p.d);
      g_post.sm = sg;
      sg += p.d;
    }
    if (p.pre) {
      copy_gain(sg, p.x.gamma_pre, p.d);
      g_pre.sm = sg;
    }
  }
  __syncthreads();
  return r;
}

template <typename T, int TEAM, int NV>
__global__ void __launch_bounds__(THREADS, 1)
    res_fwd_ring_kernel(const __grid_constant__ ResArgs p, const __grid_constant__ RingArgs q) {
  __shared__ uint64_t bars[THREADS / TEAM][MAX_DEPTH];
  __shared__ float red[2][THREADS / 32][4];
  Gain g_post, g_pre;
  const Ring<TEAM> ring = ring_setup<TEAM>(p, q, bars, g_post, g_pre);
  const int tl = ring.tl, nvec = p.d >> 3, cols = ck_cols(p.d), pitch = ck_pitch(p.d);
  const long long G = (long long)gridDim.x * (THREADS / TEAM);
  const long long first = (long long)ring.team * gridDim.x + blockIdx.x;
  if (first >= p.rows) return;
  const int n_it = (int)((p.rows - first + G - 1) / G);
  if (tl == 0)
    for (int s = 0; s < min(q.depth, n_it); ++s) ring.issue(q, s, first + s * G);
  const float alpha = p.post ? *p.x.alpha : 0.f;
  int slot = 0, stage = 0;
  uint32_t phase = 0;
  for (int it = 0; it < n_it; ++it) {
    const long long r = first + it * G;
    float tok = 0.f;
    if (p.gate == LAGA_GATE_TOKEN) tok = to_f32(static_cast<const T*>(p.x.gate)[r]);
    if (!mbar_wait(&ring.bar[stage], phase, p.x.err)) return;
    const uint8_t* buf = ring.buf + stage * q.stage_bytes;
    const uint8_t *bx = buf + q.src[F_X].off, *by = buf + q.src[F_Y].off, *bg = buf + q.src[F_G].off;
    float x[NV][8];
    if (p.post) {
      float2 st = make_float2(0.f, 1.f);
      if (p.norm_post != LAGA_NORM_NONE) {
        if (p.norm_post == LAGA_NORM_LAYER) {
          float s[1] = {0.f};
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const int v = i * TEAM + tl;
            if (v < nvec) {
              float y[8];
              Vec<T>::load(by, v, y);
#pragma unroll
              for (int k = 0; k < 8; ++k) s[0] += y[k];
            }
          }
          team_sum<TEAM, 1>(s, red, ring.team, slot);
          st.x = s[0] * p.inv_d;
        }
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int v = i * TEAM + tl;
          if (v < nvec) {
            float y[8];
            Vec<T>::load(by, v, y);
#pragma unroll
            for (int k = 0; k < 8; ++k) s[0] += (y[k] - st.x) * (y[k] - st.x);
          }
        }
        team_sum<TEAM, 1>(s, red, ring.team, slot);
        st.y = 1.f / sqrtf(s[0] * p.inv_d + p.eps);
      }
      const float tok_s = p.gate == LAGA_GATE_TOKEN ? sigmoid_pair(tok).x : 1.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = i * TEAM + tl;
        float y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[i][k] = y[k] = 0.f;
        if (v < nvec) {
          float a[8], g[8];
          Vec<T>::load(bx, v, x[i]);
          Vec<T>::load(by, v, y);
          if (p.norm_post != LAGA_NORM_NONE) {
            g_post.load(v, g);
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) g[k] = 1.f;
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            y[k] = (y[k] - st.x) * st.y;
            g[k] *= y[k];
          }
          if (p.gate == LAGA_GATE_FULL) {
            Vec<T>::load(bg, v, a);
#pragma unroll
            for (int k = 0; k < 8; ++k) g[k] *= sigmoid_pair(a[k]).x;
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) g[k] *= tok_s;
          }
#pragma unroll
          for (int k = 0; k < 8; ++k) x[i][k] += alpha * g[k];
          Vec<T>::store(p.x.x_out, r * nvec + v, x[i]);
        }
        if (p.ckpt) quantise8(static_cast<uint8_t*>(p.x.ck_y) + r * pitch, v, cols, y);
      }
      if (p.ckpt && tl < pitch - cols - cols / CK_GROUP)
        static_cast<uint8_t*>(p.x.ck_y)[r * pitch + cols + cols / CK_GROUP + tl] = 0;
      if (tl == 0) reinterpret_cast<float2*>(p.x.stat_post)[r] = st;
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = i * TEAM + tl;
#pragma unroll
        for (int k = 0; k < 8; ++k) x[i][k] = 0.f;
        if (v < nvec) Vec<T>::load(bx, v, x[i]);
      }
    }
    // the row buffer has been read by everyone: refill it
    team_sync<TEAM>(ring.team);
    if (tl == 0 && it + q.depth < n_it) ring.issue(q, stage, r + q.depth * G);
    if (p.pre) {
      float2 st = make_float2(0.f, 1.f);
      if (p.norm_pre == LAGA_NORM_LAYER) {
        float s[1] = {0.f};
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k) s[0] += x[i][k];
        team_sum<TEAM, 1>(s, red, ring.team, slot);
        st.x = s[0] * p.inv_d;
      }
      float s[1] = {0.f};
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i * TEAM + tl < nvec)
#pragma unroll
          for (int k = 0; k < 8; ++k) s[0] += (x[i][k] - st.x) * (x[i][k] - st.x);
      team_sum<TEAM, 1>(s, red, ring.team, slot);
      st.y = 1.f / sqrtf(s[0] * p.inv_d + p.eps);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = i * TEAM + tl;
        if (v < nvec) {
          float g[8];
          g_pre.load(v, g);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            x[i][k] = (x[i][k] - st.x) * st.y;
            g[k] *= x[i][k];
          }
          Vec<T>::store(p.x.h, r * nvec + v, g);
        }
        if (p.ckpt) quantise8(static_cast<uint8_t*>(p.x.ck_x) + r * pitch, v, cols, x[i]);
      }
      if (p.ckpt && tl < pitch - cols - cols / CK_GROUP)
        static_cast<uint8_t*>(p.x.ck_x)[r * pitch + cols + cols / CK_GROUP + tl] = 0;
      if (tl == 0) reinterpret_cast<float2*>(p.x.stat_pre)[r] = st;
    }
    if (++stage == q.depth) {
      stage = 0;
      phase ^= 1;
    }
  }
}

template <typename T, int TEAM, int NV>
__global__ void __launch_bounds__(THREADS, 1)
    res_bwd_ring_kernel(const __grid_constant__ ResArgs p, const __grid_constant__ RingArgs q) {
  __shared__ uint64_t bars[THREADS / TEAM][MAX_DEPTH];
  __shared__ float red[2][THREADS / 32][4];
  Gain g_post, g_pre;
  const Ring<TEAM> ring = ring_setup<TEAM>(p, q, bars, g_post, g_pre);
  const int tl = ring.tl, nvec = p.d >> 3, cols = ck_cols(p.d);
  const long long G = (long long)gridDim.x * (THREADS / TEAM);
  const long long first = (long long)ring.team * gridDim.x + blockIdx.x;
  if (first >= p.rows) return;
  const int n_it = (int)((p.rows - first + G - 1) / G);
  if (tl == 0)
    for (int s = 0; s < min(q.depth, n_it); ++s) ring.issue(q, s, first + s * G);
  const bool gain = p.norm_post != LAGA_NORM_NONE;
  const float alpha = p.post ? *p.x.alpha : 0.f;
  float acc_post[NV][8], acc_pre[NV][8], d_alpha = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < 8; ++k) acc_post[i][k] = acc_pre[i][k] = 0.f;
  int slot = 0, stage = 0;
  uint32_t phase = 0;
  for (int it = 0; it < n_it; ++it) {
    const long long r = first + it * G;
    float tok = 0.f;
    float2 st_pre = make_float2(0.f, 0.f), st_post = st_pre;
    if (p.gate == LAGA_GATE_TOKEN) tok = to_f32(static_cast<const T*>(p.x.gate)[r]);
    if (p.pre) st_pre = reinterpret_cast<const float2*>(p.x.stat_pre)[r];
    if (p.post) st_post = reinterpret_cast<const float2*>(p.x.stat_post)[r];
    if (!mbar_wait(&ring.bar[stage], phase, p.x.err)) return;
    const uint8_t* buf = ring.buf + stage * q.stage_bytes;
    const uint8_t *bd = buf + q.src[B_D].off, *bh = buf + q.src[B_DH].off;
    const uint8_t *bx = buf + q.src[B_X].off, *by = buf + q.src[B_Y].off, *bg = buf + q.src[B_G].off;
    float m0 = 0.f, m1 = 0.f;
    if (p.pre) {
      float s[2] = {0.f, 0.f};
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = i * TEAM + tl;
        if (v < nvec) {
          float dh[8], xh[8], g[8];
          Vec<T>::load(bh, v, dh);
          kept8<T>(bx, p.ckpt, cols, v, st_pre, xh);
          g_pre.load(v, g);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            acc_pre[i][k] += dh[k] * xh[k];
            const float e = dh[k] * g[k];
            s[0] += e;
            s[1] += e * xh[k];
          }
        }
      }
      team_sum<TEAM, 2>(s, red, ring.team, slot);
      m0 = p.norm_pre == LAGA_NORM_LAYER ? s[0] * p.inv_d : 0.f;
      m1 = s[1] * p.inv_d;
    }
    float f[NV][8], s[4] = {0.f, 0.f, 0.f, 0.f};   // sums: f, f y^, dx s z, token gate
    float2 tok_s = make_float2(1.f, 0.f);
    if (p.gate == LAGA_GATE_TOKEN) tok_s = sigmoid_pair(tok);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = i * TEAM + tl;
#pragma unroll
      for (int k = 0; k < 8; ++k) f[i][k] = 0.f;
      if (v < nvec) {
        float D[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) D[k] = 0.f;
        if (p.x.dx_out) Vec<T>::load(bd, v, D);
        if (p.pre) {
          float dh[8], xh[8], g[8];
          Vec<T>::load(bh, v, dh);
          kept8<T>(bx, p.ckpt, cols, v, st_pre, xh);
          g_pre.load(v, g);
#pragma unroll
          for (int k = 0; k < 8; ++k) D[k] += st_pre.y * (dh[k] * g[k] - m0 - xh[k] * m1);
          Vec<T>::store(p.x.dx, r * nvec + v, D);
        }
        if (p.post) {
          float y[8], g[8], da[8];
          kept8<T>(by, p.ckpt, cols, v, st_post, y);
          if (gain) {
            g_post.load(v, g);
          } else {
#pragma unroll
            for (int k = 0; k < 8; ++k) g[k] = 1.f;
          }
          if (p.gate == LAGA_GATE_FULL) Vec<T>::load(bg, v, da);
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float2 sg = p.gate == LAGA_GATE_FULL ? sigmoid_pair(da[k]) : tok_s;
            const float z = y[k] * g[k], dz = alpha * D[k] * sg.x;
            s[2] += D[k] * sg.x * z;
            da[k] = dz * sg.y * z;
            s[3] += da[k];
            acc_post[i][k] += dz * y[k];
            f[i][k] = dz * g[k];
            s[0] += f[i][k];
            s[1] += f[i][k] * y[k];
          }
          if (p.gate == LAGA_GATE_FULL) Vec<T>::store(p.x.dgate, r * nvec + v, da);
        }
      }
    }
    if (p.post) {
      team_sum<TEAM, 4>(s, red, ring.team, slot);
      d_alpha += s[2];
      if (p.gate == LAGA_GATE_TOKEN && tl == 0) static_cast<T*>(p.x.dgate)[r] = from_f32<T>(s[3]);
      m0 = p.norm_post == LAGA_NORM_LAYER ? s[0] * p.inv_d : 0.f;
      m1 = s[1] * p.inv_d;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = i * TEAM + tl;
        if (v < nvec) {
          if (gain) {
            float y[8];
            kept8<T>(by, p.ckpt, cols, v, st_post, y);
#pragma unroll
            for (int k = 0; k < 8; ++k) f[i][k] = st_post.y * (f[i][k] - m0 - y[k] * m1);
          }
          Vec<T>::store(p.x.dy, r * nvec + v, f[i]);
        }
      }
    }
    team_sync<TEAM>(ring.team);
    if (tl == 0 && it + q.depth < n_it) ring.issue(q, stage, r + q.depth * G);
    if (++stage == q.depth) {
      stage = 0;
      phase ^= 1;
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = i * TEAM + tl;
    if (v < nvec) {
      if (p.post && gain) Vec<float>::store(p.part_post + first * p.d, v, acc_post[i]);
      if (p.pre) Vec<float>::store(p.part_pre + first * p.d, v, acc_pre[i]);
    }
  }
  if (p.post && tl == 0) p.part_alpha[first] = d_alpha;
}

// ---------------------------------------------------------------- host side
struct Shape {
  int team, nv;
};
// Teams by width, smallest first.  The forward keeps 8 NV row values in
// registers, the backward 24 NV (two column sums and f), so its teams are
// larger for the same width.
constexpr Shape FWD_SHAPES[] = {{32, 1}, {32, 4}, {128, 4}, {256, 4}, {512, 4}};
constexpr Shape BWD_SHAPES[] = {{32, 1}, {32, 2}, {128, 2}, {256, 2}, {512, 2}, {512, 4}};

struct RingPlan {
  int team = 0, nv = 0, depth = 0;
  uint32_t gain_bytes = 0;
  uint32_t row_bytes[5] = {};
};

// The smallest team whose rings hold two rows each (one row buffer is worked
// on, the other filled), else the smallest that holds one; team 0: none does.
RingPlan ring_plan(const laga_res_dims& d, bool bwd) {
  RingPlan best;
  if (d.d % 8) return best;
  const uint32_t row = (uint32_t)d.d * (d.io_dtype == LAGA_FP32 ? 4 : 2);
  const uint32_t kept = d.ckpt ? (uint32_t)ck_pitch(d.d) : row;
  const bool gate = d.post && d.gate == LAGA_GATE_FULL;
  const uint32_t f[5] = {row, d.post ? row : 0, gate ? row : 0, 0, 0};
  const uint32_t b[5] = {row, d.pre ? row : 0, d.pre ? kept : 0, d.post ? kept : 0, gate ? row : 0};
  uint32_t stage = 0;
  for (int i = 0; i < 5; ++i) stage += bwd ? b[i] : f[i];
  const uint32_t gains =
      (uint32_t)d.d * 4 * ((d.pre ? 1 : 0) + (d.post && d.norm_post != LAGA_NORM_NONE ? 1 : 0));
  const Shape* sh = bwd ? BWD_SHAPES : FWD_SHAPES;
  const int n = bwd ? (int)(sizeof(BWD_SHAPES) / sizeof(Shape)) : (int)(sizeof(FWD_SHAPES) / sizeof(Shape));
  for (const int want : {2, 1})
    for (int i = 0; i < n; ++i) {
      if (sh[i].team * sh[i].nv * 8 < d.d) continue;
      const uint32_t all = (uint32_t)(THREADS / sh[i].team) * stage;
      for (const uint32_t g : {gains, 0u}) {
        if (g >= (uint32_t)SMEM_MAX) continue;
        const int depth = (int)std::min<uint32_t>(MAX_DEPTH, (SMEM_MAX - g) / all);
        if (depth < want) continue;
        best.team = sh[i].team;
        best.nv = sh[i].nv;
        best.depth = depth;
        best.gain_bytes = g;
        for (int k = 0; k < 5; ++k) best.row_bytes[k] = bwd ? b[k] : f[k];
        return best;
      }
    }
  return best;
}

int ring_grid(const laga_res_dims& d) { return std::min(d.rows, kSms); }

// dx_out may be missing: its place in the row buffer then stays unread
RingArgs ring_args(const RingPlan& pl, const void* const (&base)[5]) {
  RingArgs q{};
  q.depth = pl.depth;
  q.gain_bytes = pl.gain_bytes;
  uint32_t off = 0;
  for (int i = 0; i < 5; ++i) {
    q.src[i].off = off;
    q.src[i].base = static_cast<const uint8_t*>(base[i]);
    q.src[i].row_bytes = base[i] ? pl.row_bytes[i] : 0;
    off += q.src[i].row_bytes;
  }
  q.stage_bytes = off;
  return q;
}

using Kernel = void (*)(ResArgs, RingArgs);

template <typename T>
Kernel fwd_kernel(int team, int nv) {
  if (team == 32) return nv == 1 ? res_fwd_ring_kernel<T, 32, 1> : res_fwd_ring_kernel<T, 32, 4>;
  if (team == 128) return res_fwd_ring_kernel<T, 128, 4>;
  if (team == 256) return res_fwd_ring_kernel<T, 256, 4>;
  return res_fwd_ring_kernel<T, 512, 4>;
}
template <typename T>
Kernel bwd_kernel(int team, int nv) {
  if (team == 32) return nv == 1 ? res_bwd_ring_kernel<T, 32, 1> : res_bwd_ring_kernel<T, 32, 2>;
  if (team == 128) return res_bwd_ring_kernel<T, 128, 2>;
  if (team == 256) return res_bwd_ring_kernel<T, 256, 2>;
  return nv == 2 ? res_bwd_ring_kernel<T, 512, 2> : res_bwd_ring_kernel<T, 512, 4>;
}

cudaError_t launch(const char* name, Kernel k, const RingPlan& pl, const RingArgs& q,
                   const laga_res_dims& d, const ResArgs& a, cudaStream_t st) {
  const size_t smem = pl.gain_bytes + (size_t)(THREADS / pl.team) * pl.depth * q.stage_bytes;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  LaunchScope ls_(name, st);
  k<<<ring_grid(d), THREADS, smem, st>>>(a, q);
  return cudaGetLastError();
}

}  // namespace

bool ring_ok(const laga_res_dims& d, bool bwd) { return ring_plan(d, bwd).team != 0; }

int ring_slots(const laga_res_dims& d) {
  return std::min(d.rows, ring_grid(d) * (THREADS / ring_plan(d, true).team));
}

cudaError_t launch_ring_fwd(const laga_res_dims& d, const ResArgs& a, cudaStream_t st) {
  const RingPlan pl = ring_plan(d, false);
  const void* base[5] = {a.x.x, d.post ? a.x.y : nullptr,
                         a.gate == LAGA_GATE_FULL ? a.x.gate : nullptr, nullptr, nullptr};
  const Kernel k = d.io_dtype == LAGA_FP32 ? fwd_kernel<float>(pl.team, pl.nv)
                                           : fwd_kernel<__nv_bfloat16>(pl.team, pl.nv);
  return launch("res_fwd", k, pl, ring_args(pl, base), d, a, st);
}

cudaError_t launch_ring_bwd(const laga_res_dims& d, const ResArgs& a, cudaStream_t st) {
  const RingPlan pl = ring_plan(d, true);
  const void* base[5] = {a.x.dx_out, d.pre ? a.x.dh : nullptr, d.pre ? a.x.kept_x : nullptr,
                         d.post ? a.x.kept_y : nullptr,
                         a.gate == LAGA_GATE_FULL ? a.x.gate : nullptr};
  const Kernel k = d.io_dtype == LAGA_FP32 ? bwd_kernel<float>(pl.team, pl.nv)
                                           : bwd_kernel<__nv_bfloat16>(pl.team, pl.nv);
  return launch("res_bwd", k, pl, ring_args(pl, base), d, a, st);
}

}  // namespace laga
