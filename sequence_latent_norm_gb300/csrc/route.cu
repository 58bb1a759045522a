// Routing to experts (include/laga.h: laga_route_fwd, laga_route_bwd).
//
// Forward, one warp per token, expert e = 32 i + lane in register i of a lane:
// scores, the groups' two best, and top_k rounds of a warp-wide maximum.  The
// order of close scores must not depend on how a score was rounded, so every
// decision is checked: the choice runs in fp32, and where the distance between
// two neighbours of the order is within what fp32 may have lost, the token's
// choice runs again in fp64.  (Equal logits under equal biases are equal in
// both, and no reason to.)  Normal logits of 256 experts take the second run
// in about one token of 10^4; a batch of which every token takes it costs 2
// operations a clock and SM, the fp64 rate of this part.
//
// The order of the rows: a block counts its chunk's rows by expert; the second
// kernel (the same one, where the batch is one chunk) adds up the chunks in
// front of its own, and numbers its pairs in order.  Counts are integers, so
// nothing depends on the order in which blocks run.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"
#include "ops.h"

namespace laga {
namespace {

constexpr unsigned ALL = 0xffffffffu;
constexpr float TINY = 1e-20f;          // keeps the sum of a token's scores from zero

struct RouteParams {
  int tokens, experts, top_k, groups, top_groups, group_size;
  int sigmoid, renormalise;
  float scale;
  int first, local, align;
  int chunk, chunks;                     // tokens of a block, blocks
  int cap;                               // rows of `pair`
  const float* bias;
  int *expert, *row, *pair, *start;
  float* weight;
  unsigned* counts;                      // [chunks, local]
};

template <typename F> LAGA_DEVINL F minus_inf();
template <> LAGA_DEVINL float minus_inf<float>() { return __int_as_float(0xff800000); }
template <> LAGA_DEVINL double minus_inf<double>() { return __longlong_as_double(0xfff0000000000000LL); }

LAGA_DEVINL float exp_of(float x) { return expf(x); }
LAGA_DEVINL double exp_of(double x) { return exp(x); }

template <typename F>
LAGA_DEVINL F warp_add(F v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(ALL, v, o);
  return v;
}
LAGA_DEVINL float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(ALL, v, o));
  return v;
}

// One lane's part of a token: its experts' logits and biases.
template <int NV>
struct Lane {
  float l[NV], b[NV];
};

// The best of the values that a lane still has, with what belongs to it.
template <typename F>
struct Best {
  F v, s;
  float l, b;
  int e;
};

// Value and expert of the warp's best, the lowest expert of equal ones.
LAGA_DEVINL void warp_best(float v, int e, float& bv, int& be) {
  const unsigned u = __float_as_uint(v);
  const unsigned key = u & 0x80000000u ? ~u : u | 0x80000000u;
  const unsigned top = __reduce_max_sync(ALL, key);
  bv = __uint_as_float(top & 0x80000000u ? top & 0x7fffffffu : ~top);
  be = (int)__reduce_min_sync(ALL, key == top ? (unsigned)e : 0x7fffffffu);
}
LAGA_DEVINL void warp_best(double v, int e, double& bv, int& be) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const double w = __shfl_xor_sync(ALL, v, o);
    const int f = __shfl_xor_sync(ALL, e, o);
    if (w > v || (w == v && f < e)) {
      v = w;
      e = f;
    }
  }
  bv = v;
  be = e;
}

// The token's choice in F: lane j's expert (-1: none) and score.  False: the
// fp32 order is not certain.
template <int NV, typename F>
LAGA_DEVINL bool choose(const RouteParams& p, const Lane<NV>& x, int lane, int& expert, F& score) {
  constexpr bool CHECK = sizeof(F) == 4;
  const F ninf = minus_inf<F>();
  F s[NV], c[NV];
  float top = 0.f;
  if (!p.sigmoid) {
    top = x.l[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) top = fmaxf(top, x.l[i]);
    top = warp_max(top);
    if (!(top > minus_inf<float>())) top = 0.f;
    F z = F(0);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      s[i] = exp_of(F(x.l[i]) - F(top));
      z += s[i];
    }
    z = warp_add(z);
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] = z > F(0) ? s[i] / z : F(0);
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) s[i] = F(1) / (F(1) + exp_of(-F(x.l[i])));
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    c[i] = s[i] + F(x.b[i]);
    if (x.l[i] == minus_inf<float>() || !(c[i] > ninf)) c[i] = ninf;
  }
  bool sure = true;
  if (p.top_groups < p.groups) {
    F mine = ninf;                       // lane g: the score of group g
    for (int g = 0; g < p.groups; ++g) {
      const int e0 = g * p.group_size, e1 = e0 + p.group_size;
      F a = ninf, b = ninf;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = 32 * i + lane;
        if (e >= e0 && e < e1) {
          if (c[i] > a) {
            b = a;
            a = c[i];
          } else if (c[i] > b) {
            b = c[i];
          }
        }
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        const F a2 = __shfl_xor_sync(ALL, a, o), b2 = __shfl_xor_sync(ALL, b, o);
        b = a > a2 ? (b > a2 ? b : a2) : (a > b2 ? a : b2);
        a = a > a2 ? a : a2;
      }
      if (lane == g) mine = b > ninf ? a + b : a;
    }
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
      const F other = __shfl_sync(ALL, mine, g);
      rank += other > mine || (other == mine && g < lane);
    }
    if (lane >= p.groups) rank = 64;
    const unsigned keep = __ballot_sync(ALL, rank < p.top_groups);
    if (CHECK) {
      const F in = __shfl_sync(ALL, mine, __ffs(__ballot_sync(ALL, rank == p.top_groups - 1)) - 1);
      const F out = __shfl_sync(ALL, mine, __ffs(__ballot_sync(ALL, rank == p.top_groups)) - 1);
      // each of the four scores is within 2^-22, each sum within 2^-24 of itself
      const F tol = F(2.f + fabsf(float(in)) + fabsf(float(out))) * F(0x1p-20f);
      sure = !(out > ninf) || in - out > tol;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (!(keep >> ((32 * i + lane) / p.group_size) & 1u)) c[i] = ninf;
  }
  Best<F> best;
  auto rescan = [&] {
    best = Best<F>{c[0], s[0], x.l[0], x.b[0], lane};
#pragma unroll
    for (int i = 1; i < NV; ++i)
      if (c[i] > best.v) best = Best<F>{c[i], s[i], x.l[i], x.b[i], 32 * i + lane};
  };
  rescan();
  expert = -1;
  score = F(0);
  Best<F> last{};
  for (int j = 0; j < p.top_k + (CHECK ? 1 : 0); ++j) {
    Best<F> now;
    warp_best(best.v, best.e, now.v, now.e);
    if (!(now.v > ninf)) break;
    const int owner = now.e & 31;
    now.s = __shfl_sync(ALL, best.s, owner);
    if (CHECK) {
      now.l = __shfl_sync(ALL, best.l, owner);
      now.b = __shfl_sync(ALL, best.b, owner);
      if (j > 0 && !(now.l == last.l && now.b == last.b)) {
        // a score is off by 8 units in its last place, and where it is the
        // exponential of a rounded difference by that rounding; its sum by one
        const float range = p.sigmoid ? 0.f : top - now.l;
        const float tol = (float(now.s) + float(last.s)) * (16.f + 2.f * range) * 0x1p-24f +
                          (fabsf(float(now.v)) + fabsf(float(last.v))) * 0x1p-22f;
        sure = sure && float(last.v) - float(now.v) > tol;
      }
      last = now;
    }
    if (j < p.top_k && lane == j) {
      expert = now.e;
      score = now.s;
    }
    if (lane == owner) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (32 * i + lane == now.e) c[i] = ninf;
      rescan();
    }
  }
  return sure;
}

// Numbers the pairs of this block's chunk.  counts: the chunks' rows by local
// expert; smem: [experts' bases | next starts | warps x local 16-bit counts].
LAGA_DEVINL void place(const RouteParams& p, unsigned* smem) {
  const int EL = p.local, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int warps = blockDim.x >> 5;
  unsigned* base = smem;
  unsigned* next = smem + EL;
  unsigned* hist = smem + 2 * EL;        // [warps, EL]
  for (int i = threadIdx.x; i < EL * (warps + 2); i += blockDim.x) smem[i] = 0;
  __syncthreads();
  // chunks in front of this one, and all of them; `parts` threads an expert
  const int parts = max(1, (int)blockDim.x / EL);
  for (int i = threadIdx.x; i < EL * parts; i += blockDim.x) {
    const int e = i % EL;
    unsigned before = 0, all = 0;
#pragma unroll 8
    for (int c = i / EL; c < p.chunks; c += parts) {
      const unsigned n = p.counts[(size_t)c * EL + e];
      all += n;
      before += c < (int)blockIdx.x ? n : 0;
    }
    atomicAdd(&base[e], before);
    atomicAdd(&next[e], all);
  }
  __syncthreads();
  if (warp == 0) {                       // segment starts: a scan over the experts
    unsigned carry = 0;
    for (int e0 = 0; e0 < EL; e0 += 32) {
      const int e = e0 + lane;
      const unsigned all = e < EL ? next[e] : 0;
      const unsigned room = (all + p.align - 1) / p.align * p.align;
      unsigned sum = room;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned v = __shfl_up_sync(ALL, sum, o);
        if (lane >= o) sum += v;
      }
      const unsigned at = carry + sum - room;
      if (e < EL) {
        if (blockIdx.x == 0) p.start[e] = (int)at;
        // the rows of this expert that no pair takes
        if (e % (int)gridDim.x == (int)blockIdx.x)
          for (unsigned r = at + all; r < at + room; ++r) p.pair[r] = -1;
        base[e] += at;
      }
      carry += __shfl_sync(ALL, sum, 31);
    }
    if (lane == 0) {
      if (blockIdx.x == 0) p.start[EL] = (int)carry;
      next[0] = carry;
    }
  }
  const int t0 = blockIdx.x * p.chunk, t1 = min(p.tokens, t0 + p.chunk);
  const int n = (t1 - t0) * p.top_k;
  const int share = ((n + warps - 1) / warps + 31) / 32 * 32;
  const int i0 = warp * share, i1 = min(n, i0 + share);
  const long long off = (long long)t0 * p.top_k;
  unsigned* h = hist + warp * EL;
  for (int i = i0; i < i1; i += 32) {
    const int e = i + lane < i1 ? p.expert[off + i + lane] - p.first : -1;
    const bool on = e >= 0 && e < EL;
    const unsigned same = __match_any_sync(ALL, on ? e : -1);
    if (on && lane == __ffs(same) - 1) h[e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  for (int e = threadIdx.x; e < EL; e += blockDim.x) {
    unsigned at = base[e];
    for (int w = 0; w < warps; ++w) {
      const unsigned c = hist[w * EL + e];
      hist[w * EL + e] = at;
      at += c;
    }
  }
  for (long long r = (long long)next[0] + blockIdx.x * blockDim.x + threadIdx.x; r < p.cap;
       r += (long long)gridDim.x * blockDim.x)
    p.pair[r] = -1;
  __syncthreads();
  for (int i = i0; i < i1; i += 32) {
    const bool in = i + lane < i1;
    const int e = in ? p.expert[off + i + lane] - p.first : -1;
    const bool on = e >= 0 && e < EL;
    const unsigned same = __match_any_sync(ALL, on ? e : -1);
    const unsigned at = on ? h[e] + __popc(same & ((1u << lane) - 1)) : 0;
    __syncwarp();
    if (on && lane == __ffs(same) - 1) h[e] += __popc(same);
    __syncwarp();
    if (on) p.pair[at] = (int)(off + i + lane);
    if (in) p.row[off + i + lane] = on ? (int)at : -1;
  }
}

template <int NV> constexpr int route_threads() { return NV <= 8 ? 1024 : NV == 16 ? 512 : 256; }

template <int NV, typename T>
__global__ void __launch_bounds__(route_threads<NV>())
    route_kernel(const T* __restrict__ logits, const RouteParams p) {
  extern __shared__ unsigned smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int t0 = blockIdx.x * p.chunk, t1 = min(p.tokens, t0 + p.chunk);
  for (int e = threadIdx.x; e < p.local; e += blockDim.x) smem[e] = 0;
  __syncthreads();
  Lane<NV> x;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = 32 * i + lane;
    x.b[i] = p.bias && e < p.experts ? p.bias[e] : 0.f;
  }
  for (int t = t0 + warp; t < t1; t += warps) {
    bool nan = false;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = 32 * i + lane;
      x.l[i] = e < p.experts ? to_f32(logits[(long long)t * p.experts + e]) : minus_inf<float>();
      if (isnan(x.l[i]) || isnan(x.b[i]) || (!p.sigmoid && x.l[i] > 3.402823466e38f)) {
        nan = true;                       // (a softmax with an infinity is one, too)
        x.l[i] = minus_inf<float>();
      }
    }
    nan = __any_sync(ALL, nan);
    int expert;
    float score;
    if (!choose<NV, float>(p, x, lane, expert, score)) {
      double wide;
      choose<NV, double>(p, x, lane, expert, wide);
      score = (float)wide;
    }
    const float total = warp_sum(score) + TINY;
    float w = p.scale * (p.renormalise ? score / total : score);
    if (nan) w = __int_as_float(0x7fc00000);
    if (lane < p.top_k) {
      p.expert[(long long)t * p.top_k + lane] = expert;
      p.weight[(long long)t * p.top_k + lane] = expert >= 0 ? w : 0.f;
      const int e = expert - p.first;
      if (expert >= 0 && e >= 0 && e < p.local) atomicAdd(&smem[e], 1u);
    }
  }
  __syncthreads();
  for (int e = threadIdx.x; e < p.local; e += blockDim.x)
    p.counts[(size_t)blockIdx.x * p.local + e] = smem[e];
  if (p.chunks == 1) {
    __syncthreads();
    place(p, smem);
  }
}

__global__ void __launch_bounds__(1024) route_place_kernel(const RouteParams p) {
  extern __shared__ unsigned smem[];
  place(p, smem);
}

// Backward, one warp per token.  With weights w_j = scale s_j / D, D = sum s + tiny:
// ds_j = scale (dw_j - (sum_i dw_i s_i) / D) / D (scale dw_j without the
// division), then the scores' own slope.
template <typename T>
__global__ void __launch_bounds__(256)
    route_bwd_kernel(const T* __restrict__ logits, const int* __restrict__ expert,
                     const float* __restrict__ dweight, T* __restrict__ dlogits,
                     const RouteParams p) {
  extern __shared__ float rows[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, E = p.experts;
  float* g = rows + warp * E;
  for (long long t = blockIdx.x * 8LL + warp; t < p.tokens; t += gridDim.x * 8LL) {
    const T* l = logits + t * E;
    for (int e = lane; e < E; e += 32) g[e] = 0.f;
    float top = 0.f, inv = 0.f;
    if (!p.sigmoid) {
      top = minus_inf<float>();
      for (int e = lane; e < E; e += 32) top = fmaxf(top, to_f32(l[e]));
      top = warp_max(top);
      if (!(top > minus_inf<float>())) top = 0.f;
      float z = 0.f;
      for (int e = lane; e < E; e += 32) z += expf(to_f32(l[e]) - top);
      z = warp_sum(z);
      inv = z > 0.f ? 1.f / z : 0.f;
    }
    const int e = lane < p.top_k ? expert[t * p.top_k + lane] : -1;
    const bool on = e >= 0 && e < E;
    float s = 0.f, slope = 1.f, dw = 0.f;
    if (on) {
      const float x = to_f32(l[e]);
      dw = dweight[t * p.top_k + lane];
      if (p.sigmoid) {
        const float z = expf(-fabsf(x)), q = 1.f / (1.f + z);
        s = x >= 0.f ? q : z * q;
        slope = z * q * q;
      } else {
        s = expf(x - top) * inv;
      }
    }
    float ds = dw;
    if (p.renormalise) {
      const float total = warp_sum(s) + TINY, dot = warp_sum(dw * s);
      ds = (dw - dot / total) / total;
    }
    ds = on ? p.scale * ds : 0.f;
    const float mean = p.sigmoid ? 0.f : warp_sum(ds * s);
    __syncwarp();
    for (int j = 0; j < p.top_k; ++j) {   // one after the other: an expert may come twice
      if (lane == j && on) g[e] += p.sigmoid ? ds * slope : ds;
      __syncwarp();
    }
    for (int i = lane; i < E; i += 32) {
      float d = g[i];
      if (!p.sigmoid) d = (d - mean) * (expf(to_f32(l[i]) - top) * inv);
      dlogits[t * E + i] = from_f32<T>(d);
    }
    __syncwarp();
  }
}

int route_chunk(int tokens, int warps) {
  return std::max(warps, (tokens + 151) / 152);   // one block per SM, every warp a token at least
}
int route_warps(int experts) { return experts <= 256 ? 32 : experts <= 512 ? 16 : 8; }

RouteParams make_params(const laga_route_dims& d) {
  RouteParams p{};
  p.tokens = d.tokens; p.experts = d.experts; p.top_k = d.top_k;
  p.groups = d.groups; p.top_groups = d.top_groups; p.group_size = d.experts / d.groups;
  p.sigmoid = d.score == LAGA_SCORE_SIGMOID;
  p.renormalise = d.renormalise;
  p.scale = d.scale;
  p.first = d.first; p.local = d.local; p.align = d.align;
  p.chunk = route_chunk(d.tokens, route_warps(d.experts));
  p.chunks = (d.tokens + p.chunk - 1) / p.chunk;
  p.cap = (int)route_rows(d);
  return p;
}

template <int NV>
cudaError_t launch_fwd(const RouteParams& p, bool fp32, const void* logits, cudaStream_t st) {
  constexpr int threads = route_threads<NV>();
  const size_t place_smem = (size_t)p.local * (threads / 32 + 2) * 4;
  const size_t smem = p.chunks == 1 ? place_smem : (size_t)p.local * 4;
  cudaError_t e;
  {
    LaunchScope ls_("route", st);
    if (fp32) {
      if ((e = cudaFuncSetAttribute(route_kernel<NV, float>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024)) !=
          cudaSuccess)
        return e;
      route_kernel<NV, float><<<p.chunks, threads, smem, st>>>(static_cast<const float*>(logits), p);
    } else {
      if ((e = cudaFuncSetAttribute(route_kernel<NV, __nv_bfloat16>,
                                    cudaFuncAttributeMaxDynamicSharedMemorySize, 200 * 1024)) !=
          cudaSuccess)
        return e;
      route_kernel<NV, __nv_bfloat16><<<p.chunks, threads, smem, st>>>(
          static_cast<const __nv_bfloat16*>(logits), p);
    }
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (p.chunks > 1) {
    if ((e = cudaFuncSetAttribute(route_place_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  200 * 1024)) != cudaSuccess)
      return e;
    LaunchScope ls_("route_place", st);
    route_place_kernel<<<p.chunks, 1024, (size_t)p.local * 34 * 4, st>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace

laga_status route_check(const laga_route_dims* d) {
  if (!d) return LAGA_ERR_ARG;
  if (d->tokens < 0 || d->experts < 1 || d->experts > ROUTE_MAX_EXPERTS || d->top_k < 1 ||
      d->top_k > ROUTE_MAX_K || d->groups < 1 || d->groups > 32 || d->experts % d->groups ||
      d->top_groups < 1 || d->top_groups > d->groups ||
      d->top_k > d->experts / d->groups * d->top_groups)
    return LAGA_ERR_ARG;
  if (d->score != LAGA_SCORE_SIGMOID && d->score != LAGA_SCORE_SOFTMAX) return LAGA_ERR_ARG;
  if ((d->renormalise != 0 && d->renormalise != 1) || !(d->scale - d->scale == 0.f))
    return LAGA_ERR_ARG;
  if (d->first < 0 || d->local < 1 || d->local > d->experts - d->first) return LAGA_ERR_ARG;
  if (d->align != 1 && d->align != 128) return LAGA_ERR_ARG;
  if (d->io_dtype != LAGA_BF16 && d->io_dtype != LAGA_FP32) return LAGA_ERR_ARG;
  return (long long)d->tokens * d->top_k <= 0x7fffffff && route_rows(*d) <= 0x7fffffff - 128
             ? LAGA_OK : LAGA_ERR_ARG;
}

long long route_rows(const laga_route_dims& d) {
  const long long pairs = (long long)d.tokens * std::min(d.top_k, d.local);
  const long long full = std::min<long long>(d.local, pairs);
  return (pairs + full * (d.align - 1)) / d.align * d.align;
}

size_t route_ws_bytes(const laga_route_dims& d) {
  if (d.tokens == 0) return 0;
  const RouteParams p = make_params(d);
  return ((size_t)p.chunks * p.local * 4 + 255) / 256 * 256;
}

cudaError_t launch_route_fwd(const laga_route_dims& d, const void* logits, const float* bias,
                             int* expert, float* weight, int* row, int* pair, int* start,
                             unsigned char* ws, cudaStream_t st) {
  if (d.tokens == 0) return cudaMemsetAsync(start, 0, ((size_t)d.local + 1) * 4, st);
  RouteParams p = make_params(d);
  p.bias = bias;
  p.expert = expert; p.weight = weight; p.row = row; p.pair = pair; p.start = start;
  p.counts = reinterpret_cast<unsigned*>(ws);
  const bool fp32 = d.io_dtype == LAGA_FP32;
  if (d.experts <= 32) return launch_fwd<1>(p, fp32, logits, st);
  if (d.experts <= 64) return launch_fwd<2>(p, fp32, logits, st);
  if (d.experts <= 128) return launch_fwd<4>(p, fp32, logits, st);
  if (d.experts <= 256) return launch_fwd<8>(p, fp32, logits, st);
  if (d.experts <= 512) return launch_fwd<16>(p, fp32, logits, st);
  return launch_fwd<32>(p, fp32, logits, st);
}

cudaError_t launch_route_bwd(const laga_route_dims& d, const void* logits, const int* expert,
                             const float* dweight, void* dlogits, cudaStream_t st) {
  if (d.tokens == 0) return cudaSuccess;
  const RouteParams p = make_params(d);
  const int grid = (int)std::min<long long>(((long long)d.tokens + 7) / 8, 152 * 8);
  const size_t smem = (size_t)d.experts * 8 * 4;   // at most 32 KB
  LaunchScope ls_("route_bwd", st);
  if (d.io_dtype == LAGA_FP32)
    route_bwd_kernel<float><<<grid, 256, smem, st>>>(static_cast<const float*>(logits), expert,
                                                     dweight, static_cast<float*>(dlogits), p);
  else
    route_bwd_kernel<__nv_bfloat16><<<grid, 256, smem, st>>>(
        static_cast<const __nv_bfloat16*>(logits), expert, dweight,
        static_cast<__nv_bfloat16*>(dlogits), p);
  return cudaGetLastError();
}

}  // namespace laga
