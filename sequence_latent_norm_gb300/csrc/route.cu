// Routing to experts (include/laga.h: laga_route_fwd, laga_route_bwd).
//
// Forward, one warp per token, expert e = 32 i + lane in register i of a lane:
// scores, the groups' two best, and top_k rounds of a warp-wide maximum (one
// redux.sync for the value, one for the lowest expert that has it).  The order
// of close scores must not depend on how a score was rounded, so every decision
// is checked: the choice runs in fp32, and where the distance between two
// neighbours of the order is within what fp32 may have lost, it is settled in
// fp64: that of the chosen experts and of those just below them by one score a
// lane (about a token in 1000 of random logits of 256 experts), that of groups by
// one group a lane, and what is left by going over the whole token again.
// (Equal logits under equal biases are equal in both, and no reason to.)  fp64
// runs at 2 operations a clock and SM on this part: a second run of the whole
// token costs 10 us of latency, and with one for every close score the kernel
// took 78 us for 16384 x 256, and 46 us without any; it takes some 30 us now,
// bound by its instructions, 1340 a token and warp.
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
  unsigned* counts;                      // [chunks, stride]
  int stride;                            // local, rounded up to 4
};

template <typename F> LAGA_DEVINL F minus_inf();
template <> LAGA_DEVINL float minus_inf<float>() { return __int_as_float(0xff800000); }
template <> LAGA_DEVINL double minus_inf<double>() {
  return __longlong_as_double(0xfff0000000000000LL);
}

LAGA_DEVINL float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(ALL, v, o));
  return v;
}

// A float's bits in the order of the values.
LAGA_DEVINL unsigned key_of(float v) {
  const unsigned u = __float_as_uint(v);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
LAGA_DEVINL float value_of(unsigned key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);
}
constexpr unsigned KEY_OFF = 0x007fffffu;   // of -inf

// The token's logit as the choice sees it, and whether it is a NaN (or as good
// as one: a softmax with an infinity).
template <typename T>
LAGA_DEVINL float logit_of(const RouteParams& p, const T* l, int e, float b, bool& nan) {
  float x = e < p.experts ? to_f32(l[e]) : minus_inf<float>();
  if (isnan(x) || isnan(b) || (!p.sigmoid && x > 3.402823466e38f)) {
    nan = true;
    x = minus_inf<float>();
  }
  return x;
}
LAGA_DEVINL float bias_of(const RouteParams& p, int e) {
  return p.bias && e < p.experts ? p.bias[e] : 0.f;
}

// The sum of a softmax's exponentials in 64 bits.
template <int NV>
LAGA_DEVINL double wide_sum(const float (&x)[NV], float top) {
  double z = 0.0;
#pragma unroll
  for (int i = 0; i < NV; ++i) z += exp((double)x[i] - (double)top);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(ALL, z, o);
  return z;
}
LAGA_DEVINL double wide_score(const RouteParams& p, float x, float top, double z) {
  return p.sigmoid ? 1.0 / (1.0 + exp(-(double)x)) : exp((double)x - (double)top) / z;
}

// The choice in 64 bits: lane j's expert, -1 for none.
template <int NV, typename T>
__device__ __noinline__ int choose_wide(const RouteParams& p, const T* l, int lane) {
  const double ninf = minus_inf<double>();
  double c[NV], z = 1.0;
  float x[NV], top = 0.f;
  bool nan = false;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    x[i] = logit_of(p, l, 32 * i + lane, bias_of(p, 32 * i + lane), nan);
  if (!p.sigmoid) {
    top = x[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) top = fmaxf(top, x[i]);
    top = warp_max(top);
    if (!(top > minus_inf<float>())) top = 0.f;
    z = wide_sum<NV>(x, top);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    c[i] = wide_score(p, x[i], top, z) + (double)bias_of(p, 32 * i + lane);
    if (!(x[i] > minus_inf<float>()) || !(c[i] > ninf)) c[i] = ninf;
  }
  auto best_of = [&](double v, int e, double& bv, int& be) {
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
  };
  if (p.top_groups < p.groups) {
    double mine = ninf;                    // lane g: the score of group g
    for (int g = 0; g < p.groups; ++g) {
      double a = ninf, b = ninf;
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if ((32 * i + lane) / p.group_size == g) {
          if (c[i] > a) {
            b = a;
            a = c[i];
          } else if (c[i] > b) {
            b = c[i];
          }
        }
      double first, second;
      int owner, none;
      best_of(a, lane, first, owner);
      best_of(lane == owner ? b : a, lane, second, none);
      if (lane == g) mine = second > ninf ? first + second : first;
    }
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
      const double other = __shfl_sync(ALL, mine, g);
      rank += other > mine || (other == mine && g < lane);
    }
    const unsigned keep = __ballot_sync(ALL, lane < p.groups && rank < p.top_groups);
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (!(keep >> ((32 * i + lane) / p.group_size & 31) & 1u)) c[i] = ninf;
  }
  int expert = -1;
  for (int j = 0; j < p.top_k; ++j) {
    double v = ninf, bv;
    int e = 1 << 30, be;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (c[i] > v) {
        v = c[i];
        e = 32 * i + lane;
      }
    best_of(v, e, bv, be);
    if (!(bv > ninf)) break;
    if (lane == j) expert = be;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (32 * i + lane == be) c[i] = ninf;
  }
  return expert;
}

// (The functions that settle what is close read the token's logits again: what is
// handed to them stays in registers, and they hardly ever run.)
template <int NV, typename T>
LAGA_DEVINL void logits_of(const RouteParams& p, const T* l, int lane, float (&x)[NV]) {
  bool nan = false;
#pragma unroll
  for (int i = 0; i < NV; ++i)
    x[i] = logit_of(p, l, 32 * i + lane, bias_of(p, 32 * i + lane), nan);
}

// The lanes' experts in the order of their sums in 64 bits; the ones of `all`
// lanes, of which the best top_k stay.
template <int NV, typename T>
__device__ __noinline__ int reorder_wide(const RouteParams& p, const T* l, float top, int expert,
                                         int all, int lane) {
  double z = 1.0;
  if (!p.sigmoid) {
    float x[NV];
    logits_of<NV>(p, l, lane, x);
    z = wide_sum<NV>(x, top);
  }
  double c = minus_inf<double>();
  if (expert >= 0) c = wide_score(p, to_f32(l[expert]), top, z) + (double)bias_of(p, expert);
  int rank = 0;
  for (int j = 0; j < all; ++j) {
    const double other = __shfl_sync(ALL, c, j);
    const int e = __shfl_sync(ALL, expert, j);
    rank += other > c || (other == c && e < expert);
  }
  int out = -1;
  for (int j = 0; j < all; ++j) {
    const int r = __shfl_sync(ALL, rank, j), e = __shfl_sync(ALL, expert, j);
    if (r == lane) out = e;
  }
  return out;
}

// fp32 sums of score and bias, as keys.  (Explicit roundings: the same bits
// wherever it is inlined.)
template <int NV>
LAGA_DEVINL void keys_of(const RouteParams& p, const float (&x)[NV], const float (&bias)[NV],
                         float top, float inv, unsigned (&key)[NV]) {
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float s;
    if (p.sigmoid) {
      // within (1.25 |x| + 9) 2^-24 of itself; the weight is computed again
      float e;
      asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(__fmul_rn(x[i], -1.44269504f)));
      asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(__fadd_rn(1.f, e)));
    } else {
      s = __fmul_rn(expf(x[i] - top), inv);
    }
    const float c = __fadd_rn(s, bias[i]);
    key[i] = x[i] > minus_inf<float>() && c > minus_inf<float>() ? key_of(c) : KEY_OFF;
  }
}

// The choice of groups where the last one in and the first one out are close:
// the two best of every group about there, settled in 64 bits, a group a lane.
// 0 where it is not certain which two these are.
template <int NV, typename T>
__device__ __noinline__ unsigned regroup_wide(const RouteParams& p, const T* l, float top,
                                              float inv, float mine, float in, float out,
                                              float tol, float lost, int lane) {
  float x[NV], bias[NV];
  unsigned key[NV];
  logits_of<NV>(p, l, lane, x);
#pragma unroll
  for (int i = 0; i < NV; ++i) bias[i] = bias_of(p, 32 * i + lane);
  keys_of<NV>(p, x, bias, top, inv, key);
  const bool in_range = lane < p.groups;
  const unsigned above = __ballot_sync(ALL, in_range && mine > in + tol);
  const bool about = in_range && mine <= in + tol && mine >= out - tol;
  int e1 = -1, e2 = -1;
  for (unsigned left = __ballot_sync(ALL, about); left; left &= left - 1) {
    const int g = __ffs(left) - 1;
    int e[3] = {-1, -1, -1};
    float v[3];
    for (int n = 0; n < 3; ++n) {
      unsigned best = KEY_OFF;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int f = 32 * i + lane;
        if (f / p.group_size == g && f != e[0] && f != e[1]) best = max(best, key[i]);
      }
      const unsigned first = __reduce_max_sync(ALL, best);
      v[n] = value_of(first);
      if (first == KEY_OFF) break;
      unsigned f0 = 0x7fffffffu;
#pragma unroll
      for (int i = NV - 1; i >= 0; --i) {
        const int f = 32 * i + lane;
        if (f / p.group_size == g && f != e[0] && f != e[1] && key[i] == first) f0 = f;
      }
      e[n] = (int)__reduce_min_sync(ALL, f0);
    }
    if (e[2] >= 0 && !(v[1] - v[2] > 2.f * lost + (fabsf(v[1]) + fabsf(v[2])) * 0x1p-23f))
      return 0u;
    if (lane == g) {
      e1 = e[0];
      e2 = e[1];
    }
  }
  const double z = p.sigmoid ? 1.0 : wide_sum<NV>(x, top);
  double c = minus_inf<double>();
  if (e1 >= 0) {
    c = wide_score(p, to_f32(l[e1]), top, z) + (double)bias_of(p, e1);
    if (e2 >= 0) c += wide_score(p, to_f32(l[e2]), top, z) + (double)bias_of(p, e2);
  }
  int rank = __popc(above);
  for (int g = 0; g < p.groups; ++g) {
    const double other = __shfl_sync(ALL, c, g);
    const bool rival = __shfl_sync(ALL, (int)about, g);
    rank += rival && (other > c || (other == c && g < lane));
  }
  return above | __ballot_sync(ALL, about && rank < p.top_groups);
}

// fp32 scores of the experts that the lanes have chosen (0 for none).
template <int NV, typename T>
LAGA_DEVINL float score_of(const RouteParams& p, const T* l, const float (&x)[NV], int lane,
                           int expert) {
  float top = 0.f, z = 1.f;
  if (!p.sigmoid) {
    top = x[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) top = fmaxf(top, x[i]);
    top = warp_max(top);
    z = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) z += expf(x[i] - top);
    z = warp_sum(z);
  }
  if (expert < 0) return 0.f;
  const float v = to_f32(l[expert]);
  return p.sigmoid ? 1.f / (1.f + expf(-v)) : expf(v - top) / z;
}

// The choice among the keys of this lane's experts `index` (ascending), in fp32:
// lane j's expert.  `score`: its score.  False: the order is not certain.
template <int NV, int M, typename T>
LAGA_DEVINL bool pick(const RouteParams& p, const T* l, unsigned (&key)[M], const int (&index)[M],
                      float top, float inv, float lost, int lane, int& expert, float& score) {
  const float ninf = minus_inf<float>();
  // rounds: lane j keeps the j-th best
  float value = ninf;
  expert = -1;
  int found = 0;
  auto round = [&](float least) {
    unsigned best = key[0];
#pragma unroll
    for (int i = 1; i < M; ++i) best = max(best, key[i]);
    const unsigned first = __reduce_max_sync(ALL, best);
    if (first <= KEY_OFF || !(value_of(first) >= least)) return false;
    unsigned e = 0x7fffffffu;
#pragma unroll
    for (int i = M - 1; i >= 0; --i)
      if (key[i] == first) e = index[i];
    e = __reduce_min_sync(ALL, e);
#pragma unroll
    for (int i = 0; i < M; ++i)
      if (index[i] == (int)e) key[i] = KEY_OFF;
    if (lane == found) {
      expert = (int)e;
      value = value_of(first);
    }
    ++found;
    return true;
  };
  while (found < min(p.top_k + 1, 32) && round(ninf)) {
  }
  // the chosen ones' scores, and the distance of each from the next (of the last
  // one from the best that was not chosen)
  float mine = 0.f, b = 0.f;
  auto look = [&] {
    score = 0.f;
    if (expert >= 0) {
      bool nan;
      mine = logit_of(p, l, expert, 0.f, nan);
      b = bias_of(p, expert);
      score = p.sigmoid ? 1.f / (1.f + expf(-mine)) : expf(mine - top) * inv;
    }
  };
  look();
  const unsigned next = min(lane + 1, 31);
  const float v1 = __shfl_sync(ALL, value, next), l1 = __shfl_sync(ALL, mine, next);
  const float b1 = __shfl_sync(ALL, b, next);
  const int e1 = __shfl_sync(ALL, expert, next);
  // (equal ones at the end may have others next to them that were not looked at)
  const bool equal = mine == l1 && b == b1 && lane + 1 < p.top_k;
  const bool close = lane < min(p.top_k, 31) && expert >= 0 && e1 >= 0 && !equal &&
                     !(value - v1 > 2.f * lost + (fabsf(value) + fabsf(v1)) * 0x1p-24f);
  // (A choice of 32 has no lane for the one below it, and goes over the whole token
  // again: 16384 x 256 take 857 us, 111 us with 31 choices.)
  if (__any_sync(ALL, close) || p.top_k == 32) {
    // everything that may belong to the best top_k, whose last one may have lost
    // as much as what is below it
    const int last = min(p.top_k, found) - 1;
    if (last >= 0) {
      const float least = __shfl_sync(ALL, value - 2.5f * lost - fabsf(value) * 0x1p-22f, last);
      while (found < 32 && round(least)) {
      }
      // a full warp may have left some out; infinities have no distance
      if (found == 32 || !(fabsf(least) <= 3.402823466e38f)) return false;
      look();
      expert = reorder_wide<NV, T>(p, l, top, expert, found, lane);
      if (lane >= p.top_k) expert = -1;
      look();
    }
  }
  if (lane >= p.top_k) {
    expert = -1;
    score = 0.f;
  }
  return true;
}

// v[I + i], i < N, by selections, since registers have no index.
template <int I, int N, int M>
LAGA_DEVINL unsigned element(const unsigned (&v)[M], int i) {
  if constexpr (N == 1)
    return v[I];
  else
    return i & N / 2 ? element<I + N / 2, N / 2>(v, i) : element<I, N / 2>(v, i);
}

// The choice in fp32: lane j's expert.  `score`: its score.  `reach`: no sum of
// a score and a finite bias is larger.  False: the order is not certain.
template <int NV, typename T>
LAGA_DEVINL bool choose(const RouteParams& p, const T* l, const float (&x)[NV],
                        const float (&bias)[NV], const int (&group)[NV], float reach, int lane,
                        int& expert, float& score) {
  const float ninf = minus_inf<float>();
  unsigned key[NV];
  float top = 0.f, inv = 0.f;
  if (!p.sigmoid) {
    top = x[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) top = fmaxf(top, x[i]);
    top = value_of(__reduce_max_sync(ALL, key_of(top)));
    if (!(top > ninf)) top = 0.f;
    float z = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i) z += expf(x[i] - top);
    z = warp_sum(z);
    inv = z > 0.f ? 1.f / z : 0.f;
  }
  keys_of<NV>(p, x, bias, top, inv, key);
  // What fp32 may have lost of a score.  Of a sigmoid s: (1 - s) (1.25 |x| + 4)
  // units of its last place (the exponential's error) and three roundings, no
  // more than 6 units of 2^-24 of one for any x.  Of a softmax: the rounded
  // difference's and the exponential's, and its sum's (weighted by the terms, no
  // more than log E + 2 units, and NV + 5 additions); no score is above inv.
  const float lost = (p.sigmoid ? 6.f : (20.f + NV) * inv) * 0x1p-24f;
  if (p.top_groups < p.groups) {
    float mine = ninf;                     // lane g: the score of group g
    auto two_best = [&](int g, unsigned a, unsigned b) {
      const unsigned first = __reduce_max_sync(ALL, a);
      const int owner = __ffs(__ballot_sync(ALL, a == first)) - 1;
      const unsigned second = __reduce_max_sync(ALL, lane == owner ? b : a);
      if (lane == g)
        mine = second > KEY_OFF ? value_of(first) + value_of(second) : value_of(first);
    };
    if (p.group_size == 32) {              // a register each
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (i < p.groups) two_best(i, key[i], KEY_OFF);
    } else if (p.group_size % 32 == 0) {   // whole registers
      const int regs = p.group_size / 32;
      unsigned a = KEY_OFF, b = KEY_OFF;
      int left = regs, g = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        b = max(b, min(a, key[i]));
        a = max(a, key[i]);
        if (--left == 0) {
          if (g < p.groups) two_best(g, a, b);
          ++g;
          left = regs;
          a = b = KEY_OFF;
        }
      }
    } else {
      for (int g = 0; g < p.groups; ++g) {
        const int e0 = g * p.group_size, e1 = e0 + p.group_size;
        unsigned a = KEY_OFF, b = KEY_OFF;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (32 * i + 31 < e0 || 32 * i >= e1) continue;   // the same for all lanes
          const int e = 32 * i + lane;
          const unsigned k = e >= e0 && e < e1 ? key[i] : KEY_OFF;
          b = max(b, min(a, k));
          a = max(a, k);
        }
        two_best(g, a, b);
      }
    }
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
      const float other = __shfl_sync(ALL, mine, g);
      rank += other > mine || (other == mine && g < lane);
    }
    if (lane >= p.groups) rank = 64;
    unsigned keep = __ballot_sync(ALL, rank < p.top_groups);
    const int last = __ffs(__ballot_sync(ALL, rank == p.top_groups - 1)) - 1;
    const int first_out = __ffs(__ballot_sync(ALL, rank == p.top_groups)) - 1;
    const float in = __shfl_sync(ALL, mine, last), out = __shfl_sync(ALL, mine, first_out);
    // four scores, their sums with the biases, and the sums of two
    const float tol = 4.f * lost + (4.f * reach + 4.f * (fabsf(in) + fabsf(out))) * 0x1p-24f;
    if (out > ninf && !(in - out > tol)) {
      // (an infinite sum has no distance)
      keep = fabsf(in) <= 3.402823466e38f
                 ? regroup_wide<NV, T>(p, l, top, inv, mine, in, out, tol, lost, lane) : 0u;
      if (keep == 0u) return false;
    }
    if constexpr (NV >= 2 && NV <= 16) {
      // Groups of whole registers, no more than half of which are kept: the rounds
      // go over the kept ones only.  (16384 tokens, forward, without and with: 8 groups
      // of 32, 4 kept 47 and 41 us; 4 of 64, 2 kept 43.3 and 42.2; 4 of 32, 2 kept 28.3
      // and 27.8; 16 of 32, 8 kept 79 and 73.  Of 32 registers the selections cost more
      // than the rounds save: 32 of 32, 8 kept 184 and 186; 16 of 64, 8 kept 168 and 180.)
      constexpr int H = NV / 2;
      if (p.group_size % 32 == 0 && p.top_groups * (p.group_size / 32) <= H) {
        unsigned kept = keep;                // registers; the same for all lanes
        if (p.group_size != 32) {
          kept = 0;
#pragma unroll
          for (int i = 0; i < NV; ++i) kept |= (keep >> group[i] & 1u) << i;
        }
        unsigned live[H];
        int first[H];
#pragma unroll
        for (int j = 0; j < H; ++j) {
          const int i = kept ? __ffs(kept) - 1 : 0;
          live[j] = kept ? element<0, NV>(key, i) : KEY_OFF;
          first[j] = 32 * i + lane;
          kept &= kept - 1;
        }
        return pick<NV, H, T>(p, l, live, first, top, inv, lost, lane, expert, score);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (!(keep >> group[i] & 1u)) key[i] = KEY_OFF;
  }
  int index[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) index[i] = 32 * i + lane;
  return pick<NV, NV, T>(p, l, key, index, top, inv, lost, lane, expert, score);
}

// Numbers the pairs of this block's chunk.  smem: [bases | counts | warps x counts]
// by local expert.
LAGA_DEVINL void place(const RouteParams& p, unsigned* smem) {
  const int EL = p.local, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int warps = blockDim.x >> 5;
  const int t0 = blockIdx.x * p.chunk, t1 = t0 + min(p.chunk, p.tokens - t0);
  const int n = (t1 - t0) * p.top_k;
  const int share = max(((n + warps - 1) / warps + 31) / 32 * 32, 64);
  const int busy = min(warps, (n + share - 1) / share);
  const int i0 = warp * share, i1 = min(n, i0 + share);
  const int* chosen = p.expert + (long long)t0 * p.top_k;
  int early[2];                          // its loads overlap the counting
#pragma unroll
  for (int k = 0; k < 2; ++k)
    early[k] = i0 + 32 * k + lane < i1 ? chosen[i0 + 32 * k + lane] - p.first : -1;
  unsigned* base = smem;
  unsigned* next = smem + EL;
  unsigned* hist = smem + 2 * EL;        // [warps, EL]
  if (p.chunks == 1) {                   // the counts are where `base` will be
    for (int e = threadIdx.x; e < EL; e += blockDim.x) {
      next[e] = base[e];
      base[e] = 0;
    }
    for (int i = threadIdx.x; i < EL * busy; i += blockDim.x) hist[i] = 0;
  } else {
    for (int i = threadIdx.x; i < EL * (busy + 2); i += blockDim.x) smem[i] = 0;
    __syncthreads();
    // chunks in front of this one, and all of them: a thread 4 experts of every
    // `parts`-th chunk, ten loads at a time
    const int quads = p.stride / 4, parts = max(1, (int)blockDim.x / quads);
    for (int i = threadIdx.x; i < quads * parts; i += blockDim.x) {
      const int q = i % quads;
      const uint4* src = reinterpret_cast<const uint4*>(p.counts) + q;
      uint4 before = make_uint4(0, 0, 0, 0), all = before;
      for (int c0 = i / quads; c0 < p.chunks; c0 += 10 * parts) {
        uint4 n[10];
#pragma unroll
        for (int k = 0; k < 10; ++k)
          n[k] = c0 + k * parts < p.chunks ? src[(size_t)(c0 + k * parts) * quads]
                                           : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < 10; ++k) {
          all.x += n[k].x; all.y += n[k].y; all.z += n[k].z; all.w += n[k].w;
          if (c0 + k * parts < (int)blockIdx.x) {
            before.x += n[k].x; before.y += n[k].y; before.z += n[k].z; before.w += n[k].w;
          }
        }
      }
      const unsigned b4[4] = {before.x, before.y, before.z, before.w};
      const unsigned a4[4] = {all.x, all.y, all.z, all.w};
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (4 * q + k < EL) {
          atomicAdd(&base[4 * q + k], b4[k]);
          atomicAdd(&next[4 * q + k], a4[k]);
        }
    }
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
  const long long off = (long long)t0 * p.top_k;
  auto expert_at = [&](int i) {          // of pair i + lane of the chunk
    const int k = (i - i0) / 32;
    if (k < 2) return k == 0 ? early[0] : early[1];
    return i + lane < i1 ? chosen[i + lane] - p.first : -1;
  };
  unsigned* h = hist + warp * EL;
  for (int i = i0; i < i1; i += 32) {
    const int e = expert_at(i);
    const bool on = e >= 0 && e < EL;
    const unsigned same = __match_any_sync(ALL, on ? e : -1);
    if (on && lane == __ffs(same) - 1) h[e] += __popc(same);
    __syncwarp();
  }
  __syncthreads();
  for (int e = threadIdx.x; e < EL; e += blockDim.x) {
    unsigned at = base[e];
#pragma unroll 4
    for (int w = 0; w < busy; ++w) {
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
    const int e = expert_at(i);
    const bool on = e >= 0 && e < EL;
    const unsigned same = __match_any_sync(ALL, on ? e : -1);
    const unsigned at = on ? h[e] + __popc(same & ((1u << lane) - 1)) : 0;
    __syncwarp();
    if (on && lane == __ffs(same) - 1) h[e] += __popc(same);
    __syncwarp();
    if (on) p.pair[at] = (int)(off + i + lane);
    if (in) {
      const bool none = e + p.first < 0;   // no expert was on
      p.row[off + i + lane] =
          on ? (int)at : none && isnan(p.weight[off + i + lane]) ? ROUTE_ROW_NAN : -1;
    }
  }
}

template <int NV> constexpr int route_threads() { return NV <= 8 ? 1024 : NV == 16 ? 512 : 256; }

template <int NV, typename T>
__global__ void __launch_bounds__(route_threads<NV>())
    route_kernel(const T* __restrict__ logits, const RouteParams p) {
  extern __shared__ unsigned smem[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  const int t0 = blockIdx.x * p.chunk, t1 = t0 + min(p.chunk, p.tokens - t0);
  for (int e = threadIdx.x; e < p.local; e += blockDim.x) smem[e] = 0;
  __syncthreads();
  float bias[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) bias[i] = bias_of(p, 32 * i + lane);
  bool bad_bias = false;
  float reach = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    bad_bias = bad_bias || isnan(bias[i]);
    if (fabsf(bias[i]) <= 3.402823466e38f) reach = fmaxf(reach, fabsf(bias[i]));
  }
  reach = 1.f + warp_max(reach);
  int group[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) group[i] = min((32 * i + lane) / p.group_size, 31);
  for (int t = t0 + warp; t < t1; t += warps) {
    const T* l = logits + (long long)t * p.experts;
    float x[NV], most = minus_inf<float>();   // the largest, or a NaN
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = 32 * i + lane;
      x[i] = e < p.experts ? to_f32(l[e]) : minus_inf<float>();
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(most) : "f"(x[i]));
    }
    bool nan = __any_sync(ALL, isnan(most) || bad_bias ||
                                   (!p.sigmoid && most > 3.402823466e38f));
    if (nan) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        bool off = false;
        x[i] = logit_of(p, l, 32 * i + lane, bias[i], off);
      }
    }
    int expert;
    float score;
    if (!choose<NV, T>(p, l, x, bias, group, reach, lane, expert, score)) {
      expert = choose_wide<NV, T>(p, l, lane);
      score = score_of(p, l, x, lane, expert);
    }
    const float total = warp_sum(score) + TINY;
    float w = p.scale * (p.renormalise ? score / total : score);
    if (nan) w = __int_as_float(0x7fc00000);
    if (lane < p.top_k) {
      p.expert[(long long)t * p.top_k + lane] = expert;
      p.weight[(long long)t * p.top_k + lane] = expert >= 0 || nan ? w : 0.f;
      const int e = expert - p.first;
      if (expert >= 0 && e >= 0 && e < p.local) atomicAdd(&smem[e], 1u);
    }
  }
  __syncthreads();
  if (p.chunks == 1) {
    place(p, smem);
  } else {
    for (int e = threadIdx.x; e < p.local; e += blockDim.x)
      p.counts[(size_t)blockIdx.x * p.stride + e] = smem[e];
  }
}

__global__ void __launch_bounds__(1024) route_place_kernel(const RouteParams p) {
  extern __shared__ unsigned smem[];
  place(p, smem);
}

// Backward, one warp per token.  With weights w_j = scale s_j / D, D = sum s + tiny:
// ds_j = scale (dw_j - (sum_i dw_i s_i) / D) / D (scale dw_j without the
// division), then the scores' own slope.  A NaN logit's slope is a NaN, which a
// softmax hands to the whole token.  With sigmoids the logits that were not chosen
// are read only where a choice found no expert: that is every token without any,
// and reading all of them would double the kernel's bytes.
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
    const int e = lane < p.top_k ? expert[t * p.top_k + lane] : -1;
    const bool on = e >= 0 && e < E;
    if (p.sigmoid && __any_sync(ALL, lane < p.top_k && !on)) {
      for (int i = lane; i < E; i += 32)
        g[i] = isnan(to_f32(l[i])) ? __int_as_float(0x7fc00000) : 0.f;
    } else {
      for (int i = lane; i < E; i += 32) g[i] = 0.f;
    }
    float top = 0.f, inv = 0.f;
    if (!p.sigmoid) {
      top = minus_inf<float>();
      for (int i = lane; i < E; i += 32) top = fmaxf(top, to_f32(l[i]));
      top = warp_max(top);
      if (!(top > minus_inf<float>())) top = 0.f;
      float z = 0.f;
      for (int i = lane; i < E; i += 32) z += expf(to_f32(l[i]) - top);
      z = warp_sum(z);
      inv = z == 0.f ? 0.f : 1.f / z;
    }
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
  return std::max(warps, (tokens - 1) / 152 + 1);   // one block per SM, every warp a token at least
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
  p.chunks = (d.tokens - 1) / p.chunk + 1;     // (no sum of tokens here leaves 31 bits)
  p.cap = (int)route_rows(d);
  p.stride = (d.local + 3) / 4 * 4;
  return p;
}

// Words of shared memory that place needs.
constexpr size_t place_words(int local, int warps) { return (size_t)local * (warps + 2); }

template <int NV>
cudaError_t launch_fwd(const RouteParams& p, bool fp32, const void* logits, cudaStream_t st) {
  constexpr int threads = route_threads<NV>();
  // (at most 40 KB: 1024 experts come with 8 warps)
  const size_t smem = (p.chunks == 1 ? place_words(p.local, threads / 32) : p.local) * 4;
  cudaError_t e;
  {
    LaunchScope ls_("route", st);
    if (fp32)
      route_kernel<NV, float><<<p.chunks, threads, smem, st>>>(static_cast<const float*>(logits),
                                                               p);
    else
      route_kernel<NV, __nv_bfloat16><<<p.chunks, threads, smem, st>>>(
          static_cast<const __nv_bfloat16*>(logits), p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (p.chunks > 1) {
    if ((e = allow_smem(route_place_kernel, place_words(ROUTE_MAX_EXPERTS, 32) * 4)) != cudaSuccess)
      return e;
    LaunchScope ls_("route_place", st);
    route_place_kernel<<<p.chunks, 1024, place_words(p.local, 32) * 4, st>>>(p);
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
  if (p.chunks == 1) return 0;
  return ((size_t)p.chunks * p.stride * 4 + 255) / 256 * 256;
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
