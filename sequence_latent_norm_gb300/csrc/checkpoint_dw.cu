// Weight gradient from an 8-bit checkpoint (include/laga.h: laga_ckpt_dw):
//   dw[c, j] = gamma[c] sum_t v[t, c] dy[t, j],   v = code * 2^e,
// M = channels, N = columns of dy, K = tokens, on the tensor cores.  v is a
// bf16 number exactly, so the codes are turned into bf16 operand tiles on the
// way through shared memory and never exist in 16 bits in HBM: 1 byte per
// element is read instead of 2, and no separate unpacking pass (3 bytes per
// element) runs.  An fp32 dy enters as three bf16 pieces, dy = p0 + p1 + p2
// with every piece the rest cut to 8 bits (24 significand bits in all), one after
// the other against the same v tile: three products instead of one, and
// nothing of dy is lost.
//
// Pairs of CTAs (two-CTA clusters, cta_group::2, M256 pair MMAs): CTA rank r
// holds one group of 128 channels and half of the tile's BN columns.  20 warps:
//   0       TMA producer of dy tiles        (ring of NB stages)
//   1       TMA producer of code and scale tiles (NC stages)
//   2       MMA issuer (rank 0)
//   2, 3    in rank 1: pass the decoders' arrivals on to rank 0
//   3       TMEM allocator
//   4-11    decoders: code tile -> bf16 tile (NA stages), MN-major, 128-byte
//           swizzled
//   12-19   epilogue: adds up the accumulators of a tile in registers, then
//           multiplies by gamma and stores
// Decoders and epilogue wait as whole warps and run collective instructions
// in between.  A lane whose wait gave up (the error word then says so) goes
// through the rest without waiting and without telling anyone, so that its warp
// stays whole: if it left, lanes whose wait had just succeeded would be stuck.
//
// A step is 128 tokens.  Every hand-over between warps costs a few hundred
// clocks, whatever the step's size: 16384 x 7168 x 1536 takes 306 us with steps
// of 128 tokens and 377 us with 64 (the rings as deep in tokens).  What bounds
// it is that chain of hand-overs (codes, decoded tile, MMAs, and back) over
// the three v tiles that shared memory holds: without its decoding it takes
// ~280 us, with one of eight MMAs ~260 us, and the MMAs alone would take 140
// us.  With three pieces of dy per v tile the dy loads come on top.
// A decoder turns 4 codes into bf16 with 9 integer and multiply instructions.
//
// The tensor core's fp32 accumulation drops what does not fit below the
// accumulator's last place instead of rounding it: a chain of 1024 MMAs
// (16384 tokens) came out 8.4e-6 of its value short, 50 times the error of
// rounded fp32 sums.  So a chain is 64 MMAs at most, and the epilogue warps
// add the chains in registers, rounding to nearest, while the next one fills
// the other accumulator (1.7e-7).  The products of an fp32 dy's pieces have
// more bits to lose: their chain is two steps, and the smallest piece comes
// first in each, while the accumulator is small (4.5e-7, largest piece first
// 1.1e-6, one step a chain 1.2e-7 at 9 % more time; 16384 tokens).
//
// Work split: tile counts rarely fill the 76 pairs evenly, so whole rounds of
// one tile per pair run first, and the token steps of the tiles that are left
// are dealt out evenly over all pairs.  A pair's part of such a tile is a fragment in the workspace; dw_join adds a
// tile's fragments in token order.  Which pair takes what depends on the
// sizes alone, so every run adds in the same order.
#include <limits.h>

#include <algorithm>

#include "ckpt8.cuh"
#include "common.cuh"
#include "kernels.h"
#include "ops.h"
#include "sm100.cuh"
#include "tmap.h"

namespace laga {
namespace {
using namespace sm100;

constexpr int KT = 128;                      // tokens per step
constexpr int NA = 3, NB = 2, NC = 3;        // ring stages: v tiles, dy tiles, codes
constexpr int NE = 4;                        // barriers of the v tiles (a_full, a_empty)
constexpr int BOX = KT * 64 * 2;             // KT tokens x 64 bf16
constexpr int A_BYTES = 2 * BOX;             // KT tokens x 128 channels
constexpr int B_BYTES = 2 * BOX;             // KT tokens x up to 128 columns
constexpr int CODE_BYTES = KT * CK_GROUP;
constexpr int SCALE_BYTES = KT * 16;         // 16 groups' scale bytes of each token
constexpr int C_BYTES = CODE_BYTES + SCALE_BYTES;
constexpr int B_OFF = NA * A_BYTES, C_OFF = B_OFF + NB * B_BYTES;
constexpr int SMEM_BYTES = C_OFF + NC * C_BYTES + 1024;
constexpr int THREADS = 640;
constexpr int W_DEC = 4, W_EPI = 12;         // first decoder and epilogue warp
constexpr int DEC_WARPS = W_EPI - W_DEC;
// A parity tells only neighbouring phases of a barrier apart, so a waiter has
// to see every phase of the barriers that it waits on.  Everyone does but the
// two relays, which take every other step.
static_assert(NE % 2 == 0, "a v tile's barrier belongs to one relay");
static_assert(NE > NA, "a v tile's barrier outlives it");
// Registers a thread: at launch (the most that THREADS threads can have, in
// steps of 8), and after each warpgroup's setmaxnreg.
constexpr int REG_LAUNCH = 65536 / THREADS / 8 * 8;
constexpr int REG_MISC = 32, REG_DEC = 64, REG_EPI = 160;
static_assert(W_DEC % 4 == 0 && W_EPI % 4 == 0 && THREADS % 128 == 0, "whole warpgroups");
static_assert(W_DEC * REG_MISC + (W_EPI - W_DEC) * REG_DEC + (THREADS / 32 - W_EPI) * REG_EPI <=
                  THREADS / 32 * REG_LAUNCH,
              "the epilogue's warps grow on what the others give back");
constexpr int CHAIN = 8, CHAIN_PIECES = 2;   // steps of one accumulation, bf16 and fp32 dy
constexpr int TMEM_COLS = 512, ACC_COLS = 256;
constexpr int PAIRS = 76;                    // one pair per two SMs

struct DwMaps {
  CUtensorMap codes, scales, dy;
};
struct DwParams {
  int groups, cols, d, n;
  int n_tiles, tiles;
  int pieces;              // bf16 pieces of dy, all multiplied with one v tile
  int steps;               // steps of a tile
  int chain;               // steps of one accumulation
  int rounds;              // whole rounds: one tile per pair each
  int chunk;               // steps of the left-over tiles that each pair takes
  int max_frags;           // fragments per pair
  const float* gamma;
  float *dw, *frag;
  int* err;
};

// A pair's work, piece by piece: kn steps from k0 on of tile t.  frag < 0: a
// whole tile, stored to the output.
struct Walk {
  int t, k0, kn, frag;
  int i, next_t, next_k, left;   // of the pair's share of the left-over tiles

  LAGA_DEVINL Walk(const DwParams& p, int pair) {
    const long long total = (long long)(p.tiles - p.rounds * PAIRS) * p.steps;
    const long long u = min((long long)pair * p.chunk, total);
    left = (int)min((long long)p.chunk, total - u);
    next_t = p.rounds * PAIRS + (int)(u / p.steps);
    next_k = (int)(u % p.steps);
    i = 0;
  }
  LAGA_DEVINL bool next(const DwParams& p, int pair) {
    if (i < p.rounds) {
      t = i * PAIRS + pair;
      k0 = 0;
      kn = p.steps;
      frag = -1;
    } else if (left > 0) {
      t = next_t++;
      k0 = next_k;
      kn = min(left, p.steps - k0);
      frag = pair * p.max_frags + i - p.rounds;
      next_k = 0;
      left -= kn;
    } else {
      return false;
    }
    ++i;
    return true;
  }
  // The j-th step of the piece.  Neighbouring pairs start up to seven steps
  // apart and go round: the pairs that share a dy tile would otherwise all ask
  // for the same lines at once (16384 x 7168 x 576 fp32: 368 us in step, 359 us
  // apart).
  LAGA_DEVINL int step(const DwParams& p, int j) const {
    return k0 + (j + ((t / p.n_tiles) & 7)) % kn;
  }
};

LAGA_DEVINL uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t o;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(o) : "r"(a), "r"(b));
  return o;
}

// Four codes (bytes 0-3) as bf16 pairs: lo of codes 0 and 2, hi of codes 1
// and 3.  Sign, exponent and significand moved into bf16's places stand for
// the code's value times 2^-120 (e4m3's bias is 7, bf16's 127), subnormal
// codes included; m = 2^(e + 120) makes it the value, exactly.  The pairs
// leave the channels of a word in the order 0, 2, 1, 3: channel_of undoes
// that where the accumulator's rows are stored.
LAGA_DEVINL void decode4(uint32_t w, uint32_t m, uint32_t& lo, uint32_t& hi) {
  lo = mul_bf16x2(((w << 4) & 0x07f007f0u) | ((w << 8) & 0x80008000u), m);
  hi = mul_bf16x2(((w >> 4) & 0x07f007f0u) | (w & 0x80008000u), m);
}
LAGA_DEVINL int channel_of(int m) { return (m & ~3) | (m & 1) << 1 | (m >> 1 & 1); }

// 16 codes under one scale byte as two 16-byte chunks of bf16 values.  The
// factor 2^(e + 120), e = byte - 127, has the exponent field byte + 120; past
// byte 134 (e = 7) it takes two factors, and byte 255 is a NaN.
LAGA_DEVINL void decode16(const uint4& q, uint32_t byte, uint4& a, uint4& b) {
  const bool far = byte > 134u;
  const uint32_t m = far ? 0x7f007f00u : byte * 0x00800080u + 120u * 0x00800080u;
  decode4(q.x, m, a.x, a.y);
  decode4(q.y, m, a.z, a.w);
  decode4(q.z, m, b.x, b.y);
  decode4(q.w, m, b.z, b.w);
  if (far) {
    const uint32_t n = byte == CK_NAN ? 0x7fc07fc0u : (byte - 7u) * 0x00800080u;
    a = make_uint4(mul_bf16x2(a.x, n), mul_bf16x2(a.y, n), mul_bf16x2(a.z, n), mul_bf16x2(a.w, n));
    b = make_uint4(mul_bf16x2(b.x, n), mul_bf16x2(b.y, n), mul_bf16x2(b.z, n), mul_bf16x2(b.w, n));
  }
}

// Whether a phase has completed, without waiting for it.
LAGA_DEVINL bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// A thread that copies leaves when its last copies have landed (of `it` in all,
// one per barrier), also where it or those that it feeds gave up: they must
// not arrive in shared memory that the CTA has left.
template <int N>
LAGA_DEVINL void wait_landed(uint64_t (&full)[N], uint32_t it, int* err) {
  for (uint32_t i = it > N ? it - N : 0; i < it; ++i)
    mbar_wait_each(&full[i % N], (i / N) & 1, err);
}

template <int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    ckpt_dw_kernel(const __grid_constant__ DwMaps tm, const __grid_constant__ DwParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  // Each CTA's: c_full, c_empty (codes), a_empty, b_empty, acc_full (the pair
  // MMAs' commits arrive in both).  a_full: an arrival of every decoder warp,
  // and in rank 0 one that says that rank 1's is complete.  Rank 0's: b_full
  // (both CTAs' dy bytes), acc_empty (epilogue warps of both).
  __shared__ uint64_t c_full[NC], c_empty[NC], a_full[NE], a_empty[NE], b_full[NB], b_empty[NB];
  __shared__ uint64_t acc_full[2], acc_empty[2];
  __shared__ uint32_t tmem_sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1;
  constexpr int HALF = BN / 2;               // this CTA's columns of a tile

  if (threadIdx.x == 0) {
    for (int i = 0; i < NC; ++i) {
      mbar_init(&c_full[i], 1);
      mbar_init(&c_empty[i], DEC_WARPS);
    }
    for (int i = 0; i < NE; ++i) {
      mbar_init(&a_full[i], rank == 0 ? DEC_WARPS + 1 : DEC_WARPS);
      mbar_init(&a_empty[i], 1);
    }
    for (int i = 0; i < NB; ++i) {
      mbar_init(&b_full[i], 1);
      mbar_init(&b_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 16);
    }
    fence_barrier_init();
  }
  if (warp == 3) {
    tmem_alloc_pair(&tmem_sh, TMEM_COLS);
    tmem_relinquish_pair();
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers exist before anything signals them
  tc_fence_after();
  const uint32_t tmem = tmem_sh;
  Walk w(p, pair);
  if (warp < W_DEC) reg_shrink<REG_MISC>();

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tm.dy);
      uint32_t it = 0;
      bool ok = true;
      while (ok && w.next(p, pair)) {
        const int n0 = (w.t % p.n_tiles) * BN + (int)rank * HALF;
        for (int j = 0; ok && j < w.kn; ++j)
          for (int s = 0; s < p.pieces; ++s, ++it) {
            const int st = it % NB;
            if (it >= NB && !mbar_wait_each(&b_empty[st], (it / NB - 1) & 1, p.err)) {
              ok = false;
              break;
            }
            uint8_t* dst = sm + B_OFF + st * B_BYTES;
            const uint32_t bar = smem_cluster_addr(&b_full[st], 0);
            constexpr int BOXES = (HALF + 63) / 64;
            if (rank == 0) mbar_arrive_expect_tx(&b_full[st], 2 * BOXES * BOX);
#pragma unroll
            for (int b = 0; b < BOXES; ++b)
              tma_load_3d_pair(dst + b * BOX, &tm.dy, bar, n0 + b * 64, w.step(p, j) * KT,
                               p.pieces - 1 - s);
          }
      }
      // Rank 0's barriers count both CTAs' bytes.  What rank 1 may have loaded
      // beyond them was let through by commits of the MMA issuer, which leaves
      // a whole wait's limit after its last one.
      if (rank == 0) wait_landed(b_full, it, p.err);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      tma_prefetch_desc(&tm.codes);
      tma_prefetch_desc(&tm.scales);
      uint32_t it = 0;
      bool ok = true;
      while (ok && w.next(p, pair)) {
        const int g = (w.t / p.n_tiles) * 2 + (int)rank;
        for (int j = 0; j < w.kn; ++j, ++it) {
          const int t0 = w.step(p, j) * KT;
          const int st = it % NC;
          if (it >= NC && !mbar_wait_each(&c_empty[st], (it / NC - 1) & 1, p.err)) {
            ok = false;
            break;
          }
          uint8_t* dst = sm + C_OFF + st * C_BYTES;
          mbar_arrive_expect_tx(&c_full[st], C_BYTES);
          tma_load_2d(dst, &tm.codes, &c_full[st], g * CK_GROUP, t0);
          tma_load_2d(dst + CODE_BYTES, &tm.scales, &c_full[st], p.cols + (g & ~15), t0);
        }
      }
      wait_landed(c_full, it, p.err);
    }
  } else if (warp == 2 && rank == 0) {
    if (lane == 0) {
      const uint32_t idesc = idesc_bf16(256, BN, 1, 1);
      uint32_t ia = 0, ib = 0, ic = 0;   // v tiles, dy tiles, chains
      bool a_ready = false, b_ready = false;   // the next ones have been seen full
      bool ok = true;
      while (ok && w.next(p, pair)) {
        for (int k0 = 0; ok && k0 < w.kn; k0 += p.chain, ++ic) {
          const int buf = ic & 1;
          if (ic >= 2 && !mbar_wait_cluster(&acc_empty[buf], ((ic >> 1) - 1) & 1, p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t dst = tmem + (uint32_t)(buf * ACC_COLS);
          const int k1 = min(k0 + p.chain, w.kn);
          for (int k = k0; ok && k < k1; ++k, ++ia) {
            if (!a_ready && !mbar_wait_each(&a_full[ia % NE], (ia / NE) & 1, p.err)) {
              ok = false;
              break;
            }
            const uint32_t alo = sdesc_lo(smem_u32(sm + ia % NA * A_BYTES), BOX);
            for (int s = 0; s < p.pieces; ++s, ++ib) {
              const int st = ib % NB;
              if (!b_ready && !mbar_wait_each(&b_full[st], (ib / NB) & 1, p.err)) {
                ok = false;
                break;
              }
              tc_fence_after();
              // ask for the next tiles now: the answers arrive while these
              // MMAs are issued
              b_ready = mbar_test(&b_full[(ib + 1) % NB], ((ib + 1) / NB) & 1);
              a_ready = mbar_test(&a_full[(ia + 1) % NE], ((ia + 1) / NE) & 1);
              const uint32_t blo = sdesc_lo(smem_u32(sm + B_OFF + st * B_BYTES), BOX);
#pragma unroll
              for (int kk = 0; kk < KT / 16; ++kk)
                mma_ss_pair(dst, sdesc_make(alo + kk * (2048 >> 4)),
                            sdesc_make(blo + kk * (2048 >> 4)), idesc,
                            (k > k0 || s > 0 || kk > 0) ? 1u : 0u);
              mma_commit_pair(&b_empty[st]);
            }
            mma_commit_pair(&a_empty[ia % NE]);
          }
          mma_commit_pair(&acc_full[buf]);
        }
      }
      // The MMAs, whose last commit covers them all, are done before the pair's
      // shared memory and TMEM are left, also where the epilogue gave up.
      if (ic > 0) mbar_wait_each(&acc_full[(ic - 1) & 1], ((ic - 1) >> 1) & 1, p.err);
    }
  } else if (warp < W_DEC) {
    // Rank 1's warps 2 and 3, a step each in turn: announce the decoded tile
    // to rank 0.  The decoders' stores are complete for this CTA; the cluster-
    // scope release that makes them so for the pair takes ~1000 clocks, which
    // the decoders would wait for and these two do not mind.
    if (lane == 0 && rank == 1) {
      const uint32_t total = (uint32_t)(p.rounds * p.steps + w.left);
      for (uint32_t it = warp & 1; it < total; it += 2) {
        if (!mbar_wait_each(&a_full[it % NE], (it / NE) & 1, p.err)) break;
        mbar_arrive_cluster(smem_cluster_addr(&a_full[it % NE], 0));
      }
    }
  } else if (warp >= W_EPI) {
    reg_grow<REG_EPI>();
    // this warp: 32 channels (TMEM lanes) and half of the tile's columns
    const int q = warp & 3, c0 = ((warp - W_EPI) >> 2) * HALF;
    uint32_t ic = 0;
    uint32_t polls = kWaitPolls;
    while (w.next(p, pair)) {
      float2 acc[HALF / 2];
#pragma unroll
      for (int j = 0; j < HALF / 2; ++j) acc[j] = make_float2(0.f, 0.f);
      for (int k0 = 0; k0 < w.kn; k0 += p.chain, ++ic) {
        const int buf = ic & 1;
        mbar_wait_or_pass(&acc_full[buf], (ic >> 1) & 1, polls, p.err);
        tc_fence_after();
#pragma unroll
        for (int j = 0; j < HALF / 16; ++j) {
          uint32_t u[16];
          tmem_ld16(tmem_addr(tmem, q, buf * ACC_COLS + c0 + j * 16), u);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            acc[8 * j + e] = __fadd2_rn(acc[8 * j + e], make_float2(__uint_as_float(u[2 * e]),
                                                                    __uint_as_float(u[2 * e + 1])));
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && polls) mbar_arrive_cluster(smem_cluster_addr(&acc_empty[buf], 0));
      }
      const int r = (int)rank * CK_GROUP + channel_of(q * 32 + lane);   // row of the pair's tile
      const int row = (w.t / p.n_tiles) * 256 + r, n0 = (w.t % p.n_tiles) * BN + c0;
      if (polls && row < p.d) {
        const float gain = p.gamma ? p.gamma[row] : 1.f;
        float* dst = w.frag >= 0 ? p.frag + ((long long)w.frag * 256 + r) * BN + c0
                                 : p.dw + (long long)row * p.n + n0;
        const int lim = w.frag >= 0 ? HALF : p.n - n0;           // columns that exist
        if (w.frag >= 0 || p.n % 4 == 0) {
#pragma unroll
          for (int j = 0; j < HALF / 4; ++j)
            if (4 * j < lim)
              reinterpret_cast<float4*>(dst)[j] =
                  make_float4(acc[2 * j].x * gain, acc[2 * j].y * gain, acc[2 * j + 1].x * gain,
                              acc[2 * j + 1].y * gain);
        } else {
#pragma unroll
          for (int j = 0; j < HALF / 2; ++j) {
            if (2 * j < lim) dst[2 * j] = acc[j].x * gain;
            if (2 * j + 1 < lim) dst[2 * j + 1] = acc[j].y * gain;
          }
        }
      }
    }
  } else if (warp >= W_DEC) {
    reg_shrink<REG_DEC>();
    // A warp takes TOK tokens of a step, a thread 16 codes (chunk c of a
    // 64-channel box) of N of them.  Eight lanes work on the tokens r and
    // r ^ 5 of an 8-token swizzle atom and four chunks of one box: their
    // 16-byte accesses hit all eight 16-byte banks, in the code tile (chunk c
    // of token r sits at c ^ r) as in the bf16 tile (chunks 2c and 2c + 1 at
    // their own index ^ r).  The next step's codes are read before this one's
    // are decoded.
    constexpr int TOK = KT / DEC_WARPS, N = TOK / 4;
    static_assert(TOK % 8 == 0, "whole swizzle atoms");
    const int dw = warp - W_DEC, c = lane & 3, box = lane >> 3 & 1;
    uint32_t src_off[2], dst_off[2], row_off[2];   // of an atom's two token pairs of this lane
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = (2 * h + (lane >> 4)) ^ (lane & 4 ? 5 : 0);   // (0, 5), (1, 4), (2, 7), (3, 6)
      const int t = dw * TOK + r;
      row_off[h] = CODE_BYTES + t * 16;
      src_off[h] = t * CK_GROUP + (((box * 4 + c) ^ r) << 4);
      dst_off[h] = box * BOX + t * 128 + (((2 * c) ^ r) << 4);
    }
    uint4 v[N];
    uint32_t byte[N];
    uint32_t base = 0;   // steps before this piece
    uint32_t polls = kWaitPolls;
    while (w.next(p, pair)) {
      const int g = ((w.t / p.n_tiles) * 2 + (int)rank) & 15;
      const uint32_t end = base + w.kn;
      auto fetch = [&](uint32_t it) {
        const int sc = it % NC;
        mbar_wait_or_pass(&c_full[sc], (it / NC) & 1, polls, p.err);
        const uint8_t* src = sm + C_OFF + sc * C_BYTES;
#pragma unroll
        for (int h = 0; h < N; ++h) {
          v[h] = *reinterpret_cast<const uint4*>(src + src_off[h & 1] + (h >> 1) * 8 * CK_GROUP);
          byte[h] = src[row_off[h & 1] + (h >> 1) * 8 * 16 + g];
        }
      };
      fetch(base);
      for (uint32_t it = base; it < end; ++it) {
        uint4 q[N];
        uint32_t e[N];
#pragma unroll
        for (int h = 0; h < N; ++h) {
          q[h] = v[h];
          e[h] = byte[h];
        }
        if (it + 1 < end) fetch(it + 1);
        if (it >= NA)
          mbar_wait_or_pass(&a_empty[(it - NA) % NE], ((it - NA) / NE) & 1, polls, p.err);
        uint8_t* dst = sm + it % NA * A_BYTES;
#pragma unroll
        for (int h = 0; h < N; ++h) {
          uint4 a, b;
          decode16(q[h], e[h], a, b);
          const uint32_t o = dst_off[h & 1] + (h >> 1) * 8 * 128;
          *reinterpret_cast<uint4*>(dst + o) = a;
          *reinterpret_cast<uint4*>(dst + (o ^ 16)) = b;
        }
        fence_proxy_async_smem();
        __syncwarp();
        // The codes are given back only here, where what was made of them has
        // been stored: an arrival can overtake loads that are still queued,
        // and the next codes then come in under them.
        if (lane == 0 && polls) {
          mbar_arrive(&c_empty[it % NC]);
          mbar_arrive(&a_full[it % NE]);
        }
      }
      base = end;
    }
  }
  // neither CTA leaves while the pair's MMAs or the other CTA's arrivals may
  // still touch its shared memory or TMEM
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, TMEM_COLS);
  }
  cluster_sync();
}

// Sums of the left-over tiles' fragments, in token order: a thread four
// columns of a row, four fragments' loads at a time.
__global__ void __launch_bounds__(256) dw_join_kernel(const DwParams p, int bn) {
  const int vecs = bn / 4;
  const int tile = blockIdx.x / vecs;                    // vecs blocks of 256 x 4 values a tile
  const int i = (blockIdx.x % vecs) * 256 + threadIdx.x;
  const int r = i / vecs, c = (i % vecs) * 4;
  const int t = p.rounds * PAIRS + tile;
  const int row = (t / p.n_tiles) * 256 + r, n0 = (t % p.n_tiles) * bn + c;
  if (row >= p.d || n0 >= p.n) return;
  const long long u0 = (long long)tile * p.steps, u1 = u0 + p.steps;
  const int pa = (int)(u0 / p.chunk), pb = (int)((u1 - 1) / p.chunk);
  // the tile is the first piece of every pair after pa
  const int ia = tile - (int)((long long)pa * p.chunk / p.steps);
  const float* src = p.frag + (long long)r * bn + c;
  const long long slot = 256LL * bn;
  float4 s = *reinterpret_cast<const float4*>(src + (pa * p.max_frags + ia) * slot);
  for (int q = pa + 1; q <= pb; q += 4) {
    float4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k)
      v[k] = q + k <= pb ? *reinterpret_cast<const float4*>(src + (q + k) * p.max_frags * slot)
                         : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      s.x += v[k].x; s.y += v[k].y; s.z += v[k].z; s.w += v[k].w;
    }
  }
  float* dst = p.dw + (long long)row * p.n + n0;
  if (p.n % 4 == 0) {
    *reinterpret_cast<float4*>(dst) = s;
  } else {
    const float v[4] = {s.x, s.y, s.z, s.w};
    for (int k = 0; k < 4 && n0 + k < p.n; ++k) dst[k] = v[k];
  }
}

// dy in bf16 with rows of np = 8 ceil(n / 8) columns: a copy (bf16) or the
// three pieces of an fp32 value, each the rest cut to bf16's 8 significand
// bits, so that the three hold all 24.
// A thread takes 8 columns; whole rows of 16-byte loads where n allows it.
template <typename T>
__global__ void __launch_bounds__(256) dy_pieces_kernel(const T* __restrict__ dy,
                                                        __nv_bfloat16* __restrict__ out,
                                                        long long rows, int n, int np) {
  const int vecs = np / 8;
  const long long total = rows * vecs;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < total; i += gridDim.x * 256LL) {
    const long long r = total <= 0x7fffffff ? (long long)((int)i / vecs) : i / vecs;
    const int c = (int)(i - r * vecs) * 8;
    float v[8];
    if (sizeof(T) == 4 && n % 4 == 0 && c + 8 <= n) {
      const float4* src = reinterpret_cast<const float4*>(dy + r * n + c);
      const float4 a = src[0], b = src[1];
      v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
      v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = c + k < n ? to_f32(dy[r * n + c + k]) : 0.f;
    }
    // towards zero: never past the largest bf16
#pragma unroll
    for (int s = 0; s < (sizeof(T) == 4 ? 3 : 1); ++s) {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const __nv_bfloat16 a = __float2bfloat16_rz(v[2 * k]), b = __float2bfloat16_rz(v[2 * k + 1]);
        w[k] = (uint32_t)__bfloat16_as_ushort(a) | (uint32_t)__bfloat16_as_ushort(b) << 16;
        v[2 * k] = fabsf(v[2 * k]) <= 3.402823466e38f ? v[2 * k] - __bfloat162float(a) : 0.f;
        v[2 * k + 1] =
            fabsf(v[2 * k + 1]) <= 3.402823466e38f ? v[2 * k + 1] - __bfloat162float(b) : 0.f;
      }
      reinterpret_cast<uint4*>(out)[s * total + i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// ---------------------------------------------------------------- host side
struct DwPlan {
  int bn = 0, pieces = 1, np = 0;
  bool convert = false, fits = false;   // fits: the step counts stay in 32 bits
  DwParams p{};
  size_t dy_bytes = 0, frag_bytes = 0;
  int frag_slots = 0;
};

size_t up1k(size_t x) { return (x + 1023) / 1024 * 1024; }

DwPlan dw_plan(int rows, int d, int n, bool fp32) {
  DwPlan pl;
  // Columns per tile: a step costs MMA time in proportion to BN, and no less
  // than a tile of 128 columns, which the decoders set the pace of; ties go to
  // the wider tile (1536 columns: 306 us in tiles of 256, 374 us of 192; 576
  // columns fit three tiles of 192).
  long long best = -1;
  for (const int bn : {256, 192, 128}) {
    const long long cost = (long long)((n + bn - 1) / bn) * std::max(2 * bn, 256);
    if (best < 0 || cost < best) {
      best = cost;
      pl.bn = bn;
    }
  }
  pl.pieces = fp32 ? 3 : 1;
  pl.np = (n + 7) / 8 * 8;
  pl.convert = fp32 || pl.np != n;
  DwParams& p = pl.p;
  p.d = d;
  p.n = n;
  p.cols = ck_cols(d);
  p.groups = p.cols / CK_GROUP;
  p.n_tiles = (n + pl.bn - 1) / pl.bn;
  p.tiles = (p.groups + 1) / 2 * p.n_tiles;
  p.steps = (int)(((long long)rows + KT - 1) / KT);
  p.chain = fp32 ? CHAIN_PIECES : CHAIN;
  p.pieces = pl.pieces;
  p.rounds = p.tiles / PAIRS;
  const long long left = (long long)(p.tiles - p.rounds * PAIRS) * p.steps;
  // (at least four steps a pair made small products 5 to 10 % slower)
  const long long chunk = std::max<long long>((left + PAIRS - 1) / PAIRS, 1);
  pl.fits = (long long)p.rounds * p.steps + chunk + p.steps <= INT_MAX;
  if (!pl.fits) return pl;
  p.chunk = (int)chunk;
  p.max_frags = p.steps ? (int)((p.chunk + p.steps - 2) / p.steps) + 1 : 0;
  pl.frag_slots = left > 0 ? (int)((left + p.chunk - 1) / p.chunk) * p.max_frags : 0;
  if (pl.convert) pl.dy_bytes = up1k((size_t)pl.pieces * rows * pl.np * 2);
  pl.frag_bytes = up1k((size_t)pl.frag_slots * 256 * pl.bn * 4);
  return pl;
}

// Byte tensor of the checkpoint rows; boxes of 128 bytes a row are swizzled.
cudaError_t byte_map(CUtensorMap* out, const void* base, uint64_t width, uint64_t rows,
                     uint64_t pitch, uint32_t box_w) {
  auto enc = tmap_encoder();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {width, rows}, str[1] = {pitch};
  const cuuint32_t box[2] = {box_w, KT}, one[2] = {1, 1};
  const CUresult r =
      enc(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, str, box, one,
          CU_TENSOR_MAP_INTERLEAVE_NONE,
          box_w == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
          CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

bool ckpt_dw_fits(int rows, int d, int n, bool fp32) { return dw_plan(rows, d, n, fp32).fits; }

size_t ckpt_dw_ws_bytes(int rows, int d, int n, bool fp32) {
  if (rows == 0) return 0;
  const DwPlan pl = dw_plan(rows, d, n, fp32);
  return pl.dy_bytes + pl.frag_bytes;
}

cudaError_t launch_ckpt_dw(int rows, int d, int n, bool fp32, const void* ck, const void* dy,
                           const float* gamma, float* dw, unsigned char* ws, int* err,
                           cudaStream_t st) {
  if (rows == 0) return cudaMemsetAsync(dw, 0, (size_t)d * n * 4, st);
  DwPlan pl = dw_plan(rows, d, n, fp32);
  DwParams& p = pl.p;
  p.gamma = gamma;
  p.err = err;
  cudaError_t e;
  const void* dyb = dy;
  if (pl.convert) {
    dyb = ws;
    const int grid = (int)std::min<long long>(((long long)rows * (pl.np / 8) + 255) / 256, 152 * 8);
    LaunchScope ls_("ckpt_dw_pieces", st);
    if (fp32)
      dy_pieces_kernel<float><<<grid, 256, 0, st>>>(static_cast<const float*>(dy),
                                                    reinterpret_cast<__nv_bfloat16*>(ws), rows, n,
                                                    pl.np);
    else
      dy_pieces_kernel<__nv_bfloat16><<<grid, 256, 0, st>>>(
          static_cast<const __nv_bfloat16*>(dy), reinterpret_cast<__nv_bfloat16*>(ws), rows, n,
          pl.np);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  p.dw = dw;
  p.frag = reinterpret_cast<float*>(ws + pl.dy_bytes);
  DwMaps tm{};
  const uint64_t pitch = ck_pitch(d);
  if ((e = byte_map(&tm.codes, ck, p.cols, rows, pitch, CK_GROUP)) != cudaSuccess) return e;
  if ((e = byte_map(&tm.scales, ck, pitch, rows, pitch, 16)) != cudaSuccess) return e;
  {
    const uint64_t ld = (uint64_t)pl.np * 2;
    uint64_t dims[3] = {(uint64_t)pl.np, (uint64_t)rows, (uint64_t)pl.pieces};
    uint64_t str[2] = {ld, ld * rows};
    uint32_t box[3] = {64, KT, 1};
    if ((e = make_tmap_bf16(&tm.dy, dyb, 3, dims, str, box)) != cudaSuccess) return e;
  }
  auto k = pl.bn == 256 ? ckpt_dw_kernel<256> : pl.bn == 192 ? ckpt_dw_kernel<192>
                                                             : ckpt_dw_kernel<128>;
  if ((e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM_BYTES)) !=
      cudaSuccess)
    return e;
  const int left = p.tiles - p.rounds * PAIRS;
  const int pairs = p.rounds > 0 ? PAIRS : pl.frag_slots / p.max_frags;
  {
    LaunchScope ls_("ckpt_dw", st);
    k<<<2 * pairs, THREADS, SMEM_BYTES, st>>>(tm, p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (left > 0) {
    LaunchScope ls_("ckpt_dw_join", st);
    dw_join_kernel<<<left * (pl.bn / 4), 256, 0, st>>>(p, pl.bn);
  }
  return cudaGetLastError();
}

}  // namespace laga

