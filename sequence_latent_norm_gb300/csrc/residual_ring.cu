// The residual stream for rows of a multiple of 8 channels (the formulas are
// in residual.cu) whose tensors fit shared memory together, one row of each:
// all but an fp32 backward of both halves with a full gate and no checkpoints
// above 11520 channels, which residual.cu takes.
//
// Per element a bf16 junction with a full gate moves 10 bytes forward and, from
// 8-bit checkpoints, 12 backward, against 36 and 73 instructions (d = 7168).
// The forward is bound by HBM (16384 x 7168: 195 us, 0.89 of the measured
// rate), the backward by the latency of its one team an SM, which meets twice a
// row with nothing to overlap (379 us, 0.64 of the rate, 1.96 of 4 instructions
// a cycle).  Above 8192 channels a thread of the backward holds four vectors and
// spills some 450 bytes: 4096 rows from checkpoints take 111 us at 8192
// channels, 226 us at 8200 and 355 us at 16384.
//
// A CTA of 512 threads per SM is cut into teams; a team walks rows, one at a
// time, and each team has a ring of row buffers in shared memory that one
// thread keeps filled with bulk copies (cp.async.bulk, one per input tensor
// and row, completion counted on the buffer's mbarrier).  So the loads of the
// next rows are in flight while a row is worked on, whatever the reductions
// in the middle of a row wait for.  Inside a row a thread owns the 8-channel
// vectors tl, tl + TEAM, ...: 16 neighbouring threads hold one checkpoint
// group.  The gains sit in shared memory for the whole launch where they fit
// beside the rings and a team has more than one row.  Column sums (the gains'
// gradients) stay in registers over all of a team's rows and are written once,
// as one partial row per team; residual.cu adds those up.
//
// A thread whose wait for a row gave up (the error word then says so) goes
// through the rest of its rows without waiting, so that it still meets its team
// at every barrier.  Where that is the thread that fills the ring, it asks for no
// further rows, and those on their way have had the whole limit of its wait: it
// asked for all of them before.
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

// 8 consecutive elements, as pairs for the packed fp32 instructions
struct V8 {
  float2 v[4];
};
LAGA_DEVINL float2 both(float a) { return make_float2(a, a); }
LAGA_DEVINL float2 mul2(float2 a, float2 b) { return __fmul2_rn(a, b); }
LAGA_DEVINL float2 add2(float2 a, float2 b) { return __fadd2_rn(a, b); }
LAGA_DEVINL float2 fma2(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }

LAGA_DEVINL void load8(const uint8_t* p, int v, V8& f, __nv_bfloat16) {
  const uint4 w = reinterpret_cast<const uint4*>(p)[v];
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int k = 0; k < 4; ++k)
    f.v[k] = make_float2(__uint_as_float(u[k] << 16), __uint_as_float(u[k] & 0xffff0000u));
}
LAGA_DEVINL void load8(const uint8_t* p, int v, V8& f, float) {
  const float4 a = reinterpret_cast<const float4*>(p)[2 * v];
  const float4 b = reinterpret_cast<const float4*>(p)[2 * v + 1];
  f.v[0] = make_float2(a.x, a.y); f.v[1] = make_float2(a.z, a.w);
  f.v[2] = make_float2(b.x, b.y); f.v[3] = make_float2(b.z, b.w);
}
LAGA_DEVINL void store8(void* p, long long v, const V8& f, __nv_bfloat16) {
  reinterpret_cast<uint4*>(p)[v] =
      make_uint4(pack_bf16(f.v[0].x, f.v[0].y), pack_bf16(f.v[1].x, f.v[1].y),
                 pack_bf16(f.v[2].x, f.v[2].y), pack_bf16(f.v[3].x, f.v[3].y));
}
LAGA_DEVINL void store8(void* p, long long v, const V8& f, float) {
  reinterpret_cast<float4*>(p)[2 * v] = make_float4(f.v[0].x, f.v[0].y, f.v[1].x, f.v[1].y);
  reinterpret_cast<float4*>(p)[2 * v + 1] = make_float4(f.v[2].x, f.v[2].y, f.v[3].x, f.v[3].y);
}

// A row's gain: in shared memory as two planes of four floats per vector, so
// that 16-byte accesses of neighbouring threads do not collide, or global.
struct Gain {
  const float *sm, *g;
  int nvec;
  LAGA_DEVINL void load(int v, V8& f) const {
    const float4 a = sm ? reinterpret_cast<const float4*>(sm)[v]
                        : __ldg(reinterpret_cast<const float4*>(g) + 2 * v);
    const float4 b = sm ? reinterpret_cast<const float4*>(sm)[nvec + v]
                        : __ldg(reinterpret_cast<const float4*>(g) + 2 * v + 1);
    f.v[0] = make_float2(a.x, a.y); f.v[1] = make_float2(a.z, a.w);
    f.v[2] = make_float2(b.x, b.y); f.v[3] = make_float2(b.z, b.w);
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
//
// Plain form: every lane sums every value, then reads all the warps' sums
// (broadcasts, independent of one another).  Shared form, for the 16 warps of
// the largest team and several values: the lanes of a warp share the values
// out first (lane l ends up with value l mod K) and then the warps' sums, ~30
// instructions instead of ~120 for four values, in a longer chain.  The
// 7168-channel backward takes 379 us with it and 410 us without; at 4096
// channels (8 warps) it takes 61 us with it and 58 us without.
template <int TEAM, int K>
LAGA_DEVINL void team_sum(float (&v)[K], float (*red)[THREADS / 32][4], int team, int& slot) {
  constexpr uint32_t ALL = 0xffffffffu;
  constexpr int NW = TEAM / 32;
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if constexpr (NW >= 16 && (K == 2 || K == 4)) {
    const bool odd = lane & 1, two = lane & 2;
    float x = (odd ? v[1] : v[0]) + __shfl_xor_sync(ALL, odd ? v[0] : v[1], 1);
    if constexpr (K == 4) {
      const float y = (odd ? v[3] : v[2]) + __shfl_xor_sync(ALL, odd ? v[2] : v[3], 1);
      x = (two ? y : x) + __shfl_xor_sync(ALL, two ? x : y, 2);
    }
#pragma unroll
    for (int o = K; o < 32; o <<= 1) x += __shfl_xor_sync(ALL, x, o);
    if (lane < K) red[slot][w][lane] = x;
    team_sync<TEAM>(team);
    x = 0.f;
#pragma unroll
    for (int i = 0; i < NW; i += 32 / K) x += red[slot][team * NW + i + lane / K][lane % K];
#pragma unroll
    for (int o = K; o < 32; o <<= 1) x += __shfl_xor_sync(ALL, x, o);
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] = __shfl_sync(ALL, x, k);
    slot ^= 1;
    return;
  }
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = warp_sum(v[k]);
  if (TEAM == 32) return;
  if (lane == 0)
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
LAGA_DEVINL void quantise8(uint8_t* row, int v, int cols, const V8& f) {
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < 4; ++k) m = ck_max(ck_max(m, f.v[k].x), f.v[k].y);
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = ck_max(m, __shfl_xor_sync(0xffffffffu, m, o));
  float inv;
  const int s = ck_scale(m, &inv);
  if (v * 8 < cols) {
    const uint32_t lo = ck_code2(f.v[0], inv) | ck_code2(f.v[1], inv) << 16;
    const uint32_t hi = ck_code2(f.v[2], inv) | ck_code2(f.v[3], inv) << 16;
    reinterpret_cast<uint2*>(row)[v] = s == CK_NAN ? make_uint2(0, 0) : make_uint2(lo, hi);
    if ((v & 15) == 0) row[cols + (v >> 4)] = (uint8_t)s;
  }
}

// One vector of a kept row: the checkpoint's values, or (kept - mean) / std.
template <typename T>
LAGA_DEVINL void kept8(const uint8_t* row, int ckpt, int cols, int v, float2 st, V8& f) {
  if (ckpt) {
    const uint2 q = reinterpret_cast<const uint2*>(row)[v];
    const float unit = ck_unit(row[cols + (v >> 4)]);
    f.v[0] = ck_value2(q.x & 0xffffu, unit);
    f.v[1] = ck_value2(q.x >> 16, unit);
    f.v[2] = ck_value2(q.y & 0xffffu, unit);
    f.v[3] = ck_value2(q.y >> 16, unit);
  } else {
    load8(row, v, f, T());
#pragma unroll
    for (int k = 0; k < 4; ++k) f.v[k] = mul2(add2(f.v[k], both(-st.x)), both(st.y));
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
  bool ok = true;
  for (int it = 0; it < n_it; ++it) {
    const long long r = first + it * G;
    float tok = 0.f;
    if (p.gate == LAGA_GATE_TOKEN) tok = to_f32(static_cast<const T*>(p.x.gate)[r]);
    ok = ok && mbar_wait_each(&ring.bar[stage], phase, p.x.err);
    const uint8_t* buf = ring.buf + stage * q.stage_bytes;
    const uint8_t *bx = buf + q.src[F_X].off, *by = buf + q.src[F_Y].off, *bg = buf + q.src[F_G].off;
    V8 x[NV];
    if (p.post) {
      float2 st = make_float2(0.f, 1.f);
      if (p.norm_post != LAGA_NORM_NONE) {
        if (p.norm_post == LAGA_NORM_LAYER) {
          float2 t = both(0.f);
#pragma unroll
          for (int i = 0; i < NV; ++i) {
            const int v = i * TEAM + tl;
            if (v < nvec) {
              V8 y;
              load8(by, v, y, T());
#pragma unroll
              for (int k = 0; k < 4; ++k) t = add2(t, y.v[k]);
            }
          }
          float s[1] = {t.x + t.y};
          team_sum<TEAM, 1>(s, red, ring.team, slot);
          st.x = s[0] * p.inv_d;
        }
        float2 t = both(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int v = i * TEAM + tl;
          if (v < nvec) {
            V8 y;
            load8(by, v, y, T());
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 c = add2(y.v[k], both(-st.x));
              t = fma2(c, c, t);
            }
          }
        }
        float s[1] = {t.x + t.y};
        team_sum<TEAM, 1>(s, red, ring.team, slot);
        st.y = 1.f / sqrtf(s[0] * p.inv_d + p.eps);
      }
      const float tok_s = p.gate == LAGA_GATE_TOKEN ? sigmoid_pair(tok).x : 1.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = i * TEAM + tl;
        V8 y;
#pragma unroll
        for (int k = 0; k < 4; ++k) x[i].v[k] = y.v[k] = both(0.f);
        if (v < nvec) {
          V8 g;
          load8(bx, v, x[i], T());
          load8(by, v, y, T());
#pragma unroll
          for (int k = 0; k < 4; ++k) y.v[k] = mul2(add2(y.v[k], both(-st.x)), both(st.y));
          if (p.norm_post != LAGA_NORM_NONE) {
            g_post.load(v, g);
#pragma unroll
            for (int k = 0; k < 4; ++k) g.v[k] = mul2(g.v[k], y.v[k]);
          } else {
            g = y;
          }
          if (p.gate == LAGA_GATE_FULL) {
            V8 a;
            load8(bg, v, a, T());
#pragma unroll
            for (int k = 0; k < 4; ++k)
              g.v[k] = mul2(g.v[k], make_float2(sigmoid_pair(a.v[k].x).x, sigmoid_pair(a.v[k].y).x));
          } else if (p.gate == LAGA_GATE_TOKEN) {
#pragma unroll
            for (int k = 0; k < 4; ++k) g.v[k] = mul2(g.v[k], both(tok_s));
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) x[i].v[k] = fma2(both(alpha), g.v[k], x[i].v[k]);
          store8(p.x.x_out, r * nvec + v, x[i], T());
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
        for (int k = 0; k < 4; ++k) x[i].v[k] = both(0.f);
        if (v < nvec) load8(bx, v, x[i], T());
      }
    }
    // The row buffer may be refilled once everyone has used what was read from
    // it (a load can still be queued behind a barrier that its thread has
    // passed): with a residual half x' has been stored by now, without one x
    // is first used by the statistics below.
    auto refill = [&] {
      team_sync<TEAM>(ring.team);
      if (ok && tl == 0 && it + q.depth < n_it) ring.issue(q, stage, r + q.depth * G);
    };
    if (p.post) refill();
    if (p.pre) {
      float2 st = make_float2(0.f, 1.f);
      if (p.norm_pre == LAGA_NORM_LAYER) {
        float2 t = both(0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
          for (int k = 0; k < 4; ++k) t = add2(t, x[i].v[k]);
        float s[1] = {t.x + t.y};
        team_sum<TEAM, 1>(s, red, ring.team, slot);
        st.x = s[0] * p.inv_d;
      }
      float2 t = both(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i * TEAM + tl < nvec)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 c = add2(x[i].v[k], both(-st.x));
            t = fma2(c, c, t);
          }
      float s[1] = {t.x + t.y};
      team_sum<TEAM, 1>(s, red, ring.team, slot);
      st.y = 1.f / sqrtf(s[0] * p.inv_d + p.eps);
      if (!p.post) refill();
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = i * TEAM + tl;
        if (v < nvec) {
          V8 g;
          g_pre.load(v, g);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x[i].v[k] = mul2(add2(x[i].v[k], both(-st.x)), both(st.y));
            g.v[k] = mul2(g.v[k], x[i].v[k]);
          }
          store8(p.x.h, r * nvec + v, g, T());
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
  V8 acc_post[NV], acc_pre[NV];
  float d_alpha = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int k = 0; k < 4; ++k) acc_post[i].v[k] = acc_pre[i].v[k] = both(0.f);
  int slot = 0, stage = 0;
  uint32_t phase = 0;
  bool ok = true;
  for (int it = 0; it < n_it; ++it) {
    const long long r = first + it * G;
    float tok = 0.f;
    float2 st_pre = make_float2(0.f, 0.f), st_post = st_pre;
    if (p.gate == LAGA_GATE_TOKEN) tok = to_f32(static_cast<const T*>(p.x.gate)[r]);
    if (p.pre) st_pre = reinterpret_cast<const float2*>(p.x.stat_pre)[r];
    if (p.post) st_post = reinterpret_cast<const float2*>(p.x.stat_post)[r];
    ok = ok && mbar_wait_each(&ring.bar[stage], phase, p.x.err);
    const uint8_t* buf = ring.buf + stage * q.stage_bytes;
    const uint8_t *bd = buf + q.src[B_D].off, *bh = buf + q.src[B_DH].off;
    const uint8_t *bx = buf + q.src[B_X].off, *by = buf + q.src[B_Y].off, *bg = buf + q.src[B_G].off;
    float m0 = 0.f, m1 = 0.f;
    // Teams up to 256 threads keep x^ and y^ from one pass over the row to the
    // next (16384 x 2048 from checkpoints: 97 us, 102 us decoding in every
    // pass); for the one large team of a CTA the registers do not reach, and
    // keeping them took a fifth longer than decoding again (379 us at 16384 x
    // 7168).
    constexpr bool KEEP = TEAM < 512;
    V8 hat[KEEP ? NV : 1];
    if (p.pre) {
      float2 t0 = both(0.f), t1 = both(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int v = i * TEAM + tl;
        if (v < nvec) {
          V8 dh, xh, g;
          load8(bh, v, dh, T());
          kept8<T>(bx, p.ckpt, cols, v, st_pre, xh);
          g_pre.load(v, g);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            acc_pre[i].v[k] = fma2(dh.v[k], xh.v[k], acc_pre[i].v[k]);
            const float2 e = mul2(dh.v[k], g.v[k]);
            t0 = add2(t0, e);
            t1 = fma2(e, xh.v[k], t1);
          }
          if (KEEP) hat[i] = xh;
        }
      }
      float s[2] = {t0.x + t0.y, t1.x + t1.y};
      team_sum<TEAM, 2>(s, red, ring.team, slot);
      m0 = p.norm_pre == LAGA_NORM_LAYER ? s[0] * p.inv_d : 0.f;
      m1 = s[1] * p.inv_d;
    }
    V8 f[NV];
    float2 t0 = both(0.f), t1 = t0, t2 = t0, t3 = t0;   // sums: f, f y^, dx s z, token gate
    float2 tok_s = make_float2(1.f, 0.f);
    if (p.gate == LAGA_GATE_TOKEN) tok_s = sigmoid_pair(tok);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int v = i * TEAM + tl;
#pragma unroll
      for (int k = 0; k < 4; ++k) f[i].v[k] = both(0.f);
      if (v < nvec) {
        V8 D;
#pragma unroll
        for (int k = 0; k < 4; ++k) D.v[k] = both(0.f);
        if (p.x.dx_out) load8(bd, v, D, T());
        if (p.pre) {
          V8 dh, xh, g;
          load8(bh, v, dh, T());
          if (KEEP)
            xh = hat[i];
          else
            kept8<T>(bx, p.ckpt, cols, v, st_pre, xh);
          g_pre.load(v, g);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 e = fma2(xh.v[k], both(-m1), fma2(dh.v[k], g.v[k], both(-m0)));
            D.v[k] = fma2(both(st_pre.y), e, D.v[k]);
          }
          store8(p.x.dx, r * nvec + v, D, T());
        }
        if (p.post) {
          V8 y, g, a;
          kept8<T>(by, p.ckpt, cols, v, st_post, y);
          if (KEEP) hat[i] = y;
          if (gain) {
            g_post.load(v, g);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) g.v[k] = both(1.f);
          }
          if (p.gate == LAGA_GATE_FULL) load8(bg, v, a, T());
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float2 s = both(tok_s.x), c = both(tok_s.y);
            if (p.gate == LAGA_GATE_FULL) {
              const float2 u = sigmoid_pair(a.v[k].x), w = sigmoid_pair(a.v[k].y);
              s = make_float2(u.x, w.x);
              c = make_float2(u.y, w.y);
            }
            const float2 Ds = mul2(D.v[k], s), z = mul2(y.v[k], g.v[k]);
            const float2 u = mul2(Ds, z), dz = mul2(both(alpha), Ds);
            t2 = add2(t2, u);
            a.v[k] = mul2(mul2(both(alpha), u), c);
            t3 = add2(t3, a.v[k]);
            acc_post[i].v[k] = fma2(dz, y.v[k], acc_post[i].v[k]);
            f[i].v[k] = mul2(dz, g.v[k]);
            t0 = add2(t0, f[i].v[k]);
            t1 = fma2(f[i].v[k], y.v[k], t1);
          }
          if (p.gate == LAGA_GATE_FULL) store8(p.x.dgate, r * nvec + v, a, T());
        }
      }
    }
    if (p.post) {
      float s[4] = {t0.x + t0.y, t1.x + t1.y, t2.x + t2.y, t3.x + t3.y};
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
            V8 y;
            if (KEEP)
              y = hat[i];
            else
              kept8<T>(by, p.ckpt, cols, v, st_post, y);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              f[i].v[k] = mul2(both(st_post.y),
                               fma2(y.v[k], both(-m1), add2(f[i].v[k], both(-m0))));
          }
          store8(p.x.dy, r * nvec + v, f[i], T());
        }
      }
    }
    // every value read from the row buffer has gone into a store by now
    team_sync<TEAM>(ring.team);
    if (ok && tl == 0 && it + q.depth < n_it) ring.issue(q, stage, r + q.depth * G);
    if (++stage == q.depth) {
      stage = 0;
      phase ^= 1;
    }
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = i * TEAM + tl;
    if (v < nvec) {
      if (p.post && gain) store8(p.part_post + first * p.d, v, acc_post[i], 0.f);
      if (p.pre) store8(p.part_pre + first * p.d, v, acc_pre[i], 0.f);
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

int ring_grid(const laga_res_dims& d) { return std::min(d.rows, kSms); }

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
        // Rows of one team.  With one, the gains would be copied for a single
        // use, and a short ring keeps a small call's shared memory small.
        const int per = ring_grid(d) ? (d.rows - 1) / (ring_grid(d) * (THREADS / sh[i].team)) + 1 : 1;
        best.depth = std::min(depth, per);
        best.gain_bytes = per > 1 ? g : 0;
        for (int k = 0; k < 5; ++k) best.row_bytes[k] = bwd ? b[k] : f[k];
        return best;
      }
    }
  return best;
}

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
  if (smem > 44 * 1024) {   // 48 KB with the static part need no opt-in
    // the limit belongs to the kernel, which other threads may be launching
    // with other sizes: it is the same in every call
    const cudaError_t e =
        cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_MAX);
    if (e != cudaSuccess) return e;
  }
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
