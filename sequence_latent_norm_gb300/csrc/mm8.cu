// Products of 8-bit rows on the tensor cores (include/laga.h: laga_mm8):
//   y[r, j] = sum_i a[r, i] b[e n + j, i]
// with e4m3 codes and one power-of-two scale per 128 of i on both sides.  The
// block-scaled MMA (kind::mxf8f6f4) takes such scales itself, one UE8M0 byte
// per 32 of i: the checkpoints' scale bytes are that format (b stands for
// 2^(b - 127), 255 for NaN), and four neighbouring MMAs (K = 32) name the same
// byte.  So codes and scales go from HBM to the tensor core as they are.
//
// M = columns of y (rows of b), N = rows of y (rows of a): a tile's N can be
// any multiple of 32, so that experts with few rows, and single tokens, cost
// what they need, and b, which is the larger operand then, is streamed through
// full 256-row tiles.
//
// Persistent pairs of CTAs (two-CTA clusters, cta_group::2): CTA rank r holds
// 128 of a tile's rows of b and half of its rows of a.  12 warps:
//   0     TMA producer of codes         (ring of STAGES, two steps of K = 128 each)
//   1     MMA issuer (rank 0), TMEM allocator
//   2     scale loader: four steps' bytes of each row, a 32-bit word, into the
//         32 x 128-bit layout that tcgen05.cp spreads over TMEM; 16 steps' words
//         at a time (ring of SF_SLOTS), since loading them and telling the other
//         CTA takes some 2500 clocks
//   4-11  epilogue: accumulator -> registers -> y (or, where K is split, fp32
//         partial sums, which mm8_join adds up in order)
// TMEM: two accumulators of up to 224 columns, so that one drains while the
// other fills, and four sets of scales.
//
// What bounds it (16384 x 7168 x 7168, bf16 out: 531 us, 3170 TFLOP/s, 0.83 of
// twice the measured bf16 rate): what stands between the MMAs, which keep the
// tensor pipe busy for 65 % of the clocks at 16384 x 7168 x 1536.  A step takes
// some 690 clocks of a pair, 448 of them its MMAs at the nominal rate; the rest are
// the waits, commits and copies of scales of the one thread that issues (with a
// wait per 128 of i instead of 256 and scales fetched 4 steps at a time 690 us), and
// loads of 45 bytes a clock into a shared memory that the MMAs read at the same
// time.  Short K (16384 x 2048 x 7168: 216 us) adds the output's 235 MB; a few rows
// are bound by b's bytes, one token by the 56 of 76 pairs that its pieces of K fill,
// and the launch that joins them (7168 x 7168: 28 us).
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

constexpr int KS = CK_GROUP;                 // codes of i per step, the swizzled width
constexpr int HALVES = 2;                    // steps per stage
constexpr int FT = 256;                      // rows of b per tile
constexpr int TN_MAX = 224;                  // rows of a per tile
constexpr int W_BYTES = 128 * KS, X_OFF = HALVES * W_BYTES;
constexpr int SF_BYTES = 3 * 512;            // 4 steps' words of 128 rows of b, 2 x 128 of a
constexpr int SF_WORDS = 4, SF_SLOTS = 2;    // such words in a slot of the ring
constexpr int SF_STEPS = 4 * SF_WORDS;
constexpr int SF_SETS = 4;                   // sets of scales in tensor memory
constexpr int SLOT_BYTES = 2048, EPI_WARPS = 8;
// Shared memory for tiles of up to TN rows of a.  With few rows, where b's bytes
// are all that counts, the ring is deeper (16 rows of 32 experts x 7168 x 4096:
// 89 us, 91 us with three stages).
template <int TN>
struct Ring {
  static constexpr int STAGES = TN > 32 ? 3 : 5;
  static constexpr int X_BYTES = TN / 2 * KS, STAGE_BYTES = X_OFF + HALVES * X_BYTES;
  static constexpr int SF_OFF = STAGES * STAGE_BYTES;
  static constexpr int OUT_OFF = SF_OFF + SF_SLOTS * SF_WORDS * SF_BYTES;
  static constexpr int SMEM_BYTES = OUT_OFF + EPI_WARPS * SLOT_BYTES + 1024;
  static_assert(SMEM_BYTES + (int)sizeof(int) * 3 * (ROUTE_MAX_EXPERTS + 1) + 1024 + 256 <=
                    228 * 1024,
                "shared memory, with the segments and the barriers");
  // A set of scales is written again SF_SETS words later, and the MMAs that read
  // it must be done by then.  Words of one tile or two have at least SF_SETS - 1
  // others between them, of two stages each but for a tile's last one, which may
  // have one: no fewer stages than the ring lets be in flight.  (Words of tiles
  // further apart have a wait for an accumulator between them.)
  static_assert((SF_SETS - 1) * (4 / HALVES) - 1 >= STAGES,
                "scales outlive the MMAs that read them");
};
constexpr int THREADS = 128 + 32 * EPI_WARPS;
constexpr int TMEM_COLS = 512, SF_COL = 2 * TN_MAX, SF_COLS = 16;
static_assert(SF_COL + SF_SETS * SF_COLS <= TMEM_COLS, "tensor memory");
static_assert(4 % HALVES == 0, "whole stages under a word of scales");
constexpr int PAIRS = 76;                    // one pair per two SMs
// Column tiles that run side by side, sharing their rows of a through L2 (16384 x
// 7168 x 7168: 576, 547 and 529 us with 4, 8 and 16).
constexpr int BAND = 16;
constexpr int WMAX = ROUTE_MAX_EXPERTS;

struct Maps {
  CUtensorMap w, x, y;
};
struct Params {
  int rows, n, experts;    // experts 0: one matrix
  int tn;                  // rows of a per tile, a multiple of 32
  int f_tiles;             // column tiles
  int steps;               // steps of the whole K
  int splits, split_steps; // pieces of K, steps of each
  int pitch, cols;         // bytes of a row of a and b, of its codes
  int bf16;
  int mapped;              // y has a tensor map
  const uint8_t *a, *b;
  const int *start, *pair;
  void* y;                 // or the partial sums [splits, rows, n]
  int* err;
};

// The experts' first rows, the ends of those that belong to pairs, and the row
// tiles in front of each.
struct Segments {
  int start[WMAX + 1], end[WMAX], tiles[WMAX + 1];
};

// A pair's tiles in turn: rows r0 .. r1 of expert e, column tile f, steps k0 ..
struct Walk {
  int t, e;                // next tile, and the expert of the last one
  int r0, r1, r2, f, k0, kn, z;   // rows r1 .. r2: of no pair, zeros

  LAGA_DEVINL explicit Walk(int pair) : t(pair), e(0) {}
  LAGA_DEVINL bool next(const Params& p, const Segments& s) {
    const int per = p.f_tiles * p.splits, E = max(p.experts, 1);
    while (e < E && t >= s.tiles[e + 1] * per) ++e;
    if (e >= E) return false;
    const int q = t - s.tiles[e] * per, tt = s.tiles[e + 1] - s.tiles[e];
    z = q % p.splits;
    const int u = q / p.splits;
    const int band = u / (BAND * tt), fb = min(BAND, p.f_tiles - band * BAND);
    const int v = u - band * BAND * tt;
    f = band * BAND + v % fb;
    r0 = s.start[e] + v / fb * p.tn;
    r1 = min(s.end[e], r0 + p.tn);
    r2 = r1 == s.end[e] ? s.start[e + 1] : r1;
    k0 = z * p.split_steps;
    kn = min(p.split_steps, p.steps - k0);
    t += gridDim.x >> 1;
    return true;
  }
  // N of the tile's MMAs
  LAGA_DEVINL int width() const { return max((r1 - r0 + 31) / 32 * 32, 32); }
};

// Block-scaled MMA: D (+)= (A scaleA) (B scaleB)^T, both CTAs of the pair.
LAGA_DEVINL void mma_mx_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                             uint32_t sfb, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::mxf8f6f4.block_scale.scale_vec::1X"
      " [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(sfa), "r"(sfb)
      : "memory");
}
// e4m3 operands, K-major, UE8M0 scales; `byte`: which of a scale word's four.
LAGA_DEVINL uint32_t idesc_mx(int n, int byte) {
  return (uint32_t)byte << 4 | (uint32_t)(n >> 3) << 17 | 1u << 23 | (uint32_t)(FT >> 4) << 24 |
         (uint32_t)byte << 29;
}
// 32 x 128 bits of shared memory into 32 lanes x 4 columns, for all four
// quadrants of lanes, in both CTAs (each from its own shared memory).
LAGA_DEVINL void copy_scales_pair(uint32_t taddr, uint32_t saddr) {
  const uint64_t desc = (uint64_t)(8u | 1u << 14) << 32 | ((saddr >> 4) & 0x3fffu);
  asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;" ::"r"(taddr), "l"(desc)
               : "memory");
}

// A thread that copies leaves when its last copies have landed.
template <int N>
LAGA_DEVINL void wait_landed(uint64_t (&full)[N], uint32_t it, int* err) {
  for (uint32_t i = it > N ? it - N : 0; i < it; ++i)
    mbar_wait_each(&full[i % N], (i / N) & 1, err);
}

// This warp's 32 columns x 32 rows of y, from the accumulator's lanes, which are
// columns here, to rows: through a slot of [rows][32 columns] in shared memory
// and a tensor store, or (a tile's last rows, widths that no tensor map takes)
// lane by lane.
template <typename T>
LAGA_DEVINL void store_rows(const Params& p, const CUtensorMap* ym, const Walk& w,
                            const float (&v)[32], int lane, int c0, int col0, uint8_t* out) {
  constexpr int R = SLOT_BYTES / (32 * sizeof(T));   // rows of a slot
  const int j = col0 + lane, n = w.r1 - w.r0;
  const long long row0 = (long long)w.z * p.rows + w.r0;
  T* dst = static_cast<T*>(p.y) + row0 * p.n + j;
#pragma unroll
  for (int h = 0; h < 32; h += R) {
    if (p.mapped && c0 + h + R <= n) {
      T* slot = reinterpret_cast<T*>(out);
      if (lane == 0) bulk_wait_read0();     // the store that last read the slot
      __syncwarp();
#pragma unroll
      for (int c = 0; c < R; ++c) slot[c * 32 + lane] = from_f32<T>(v[h + c]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        if (col0 < p.n) tma_store_2d(ym, slot, col0, (int)row0 + c0 + h);
        bulk_commit();
      }
    } else if (j < p.n) {
#pragma unroll
      for (int c = 0; c < R; ++c)
        if (c0 + h + c < n) dst[(long long)(c0 + h + c) * p.n] = from_f32<T>(v[h + c]);
    }
  }
}

// The tile's rows of no pair.
template <typename T>
LAGA_DEVINL void store_zeros(const Params& p, const Walk& w, int j) {
  T* dst = static_cast<T*>(p.y) + ((long long)w.z * p.rows + w.r1) * p.n + j;
  if (j < p.n)
    for (int r = 0; r < w.r2 - w.r1; ++r) dst[(long long)r * p.n] = from_f32<T>(0.f);
}

LAGA_DEVINL void load_rows(uint32_t taddr, float (&v)[32]) {
  uint32_t u[32];
  tmem_ld32(taddr, u);
#pragma unroll
  for (int c = 0; c < 32; ++c) v[c] = __uint_as_float(u[c]);
}

// CHAINS: y in fp32, added up in registers over chains of SF_STEPS steps.
template <int TN, bool CHAINS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    mm8_kernel(const __grid_constant__ Maps tm, const __grid_constant__ Params p) {
  constexpr int STAGES = Ring<TN>::STAGES, STAGE_BYTES = Ring<TN>::STAGE_BYTES;
  constexpr int X_BYTES = Ring<TN>::X_BYTES, SF_OFF = Ring<TN>::SF_OFF;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sm = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                           ~static_cast<uintptr_t>(1023));
  // full, sf_full, acc_empty: rank 0's, counting both CTAs; empty, sf_empty,
  // acc_full: each CTA's, by the pair MMAs' commits
  __shared__ uint64_t full[STAGES], empty[STAGES], sf_full[SF_SLOTS], sf_empty[SF_SLOTS];
  __shared__ uint64_t acc_full[2], acc_empty[2];
  __shared__ uint32_t tmem_sh;
  __shared__ Segments seg;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();

  if (threadIdx.x == 0) {
    for (int i = 0; i < STAGES; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], 1);
    }
    for (int i = 0; i < SF_SLOTS; ++i) {
      mbar_init(&sf_full[i], 2);
      mbar_init(&sf_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&acc_full[i], 1);
      mbar_init(&acc_empty[i], 2 * EPI_WARPS);
    }
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(&tmem_sh, TMEM_COLS);
    tmem_relinquish_pair();
  }
  if (warp == 2) {
    // row tiles in front of each expert: a scan, 32 experts at a time
    const int E = max(p.experts, 1);
    int carry = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      int s = 0, t = 0;
      if (e < E) {
        s = p.experts ? min(max(p.start[e], 0), p.rows) : 0;
        t = p.experts ? min(max(p.start[e + 1], 0), p.rows) : p.rows;
      }
      int end = t;
      if (p.pair) {
        // the rows of no pair are the last ones, fewer than 128
        for (int lo = max(s, t - 127); lo < end;) {
          const int mid = (lo + end) >> 1;
          if (p.pair[mid] < 0)
            end = mid;
          else
            lo = mid + 1;
        }
      }
      const int own = e < E && t > s ? max((end - s + p.tn - 1) / p.tn, 1) : 0;
      int sum = own;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += v;
      }
      if (e < E) {
        seg.start[e] = s;
        seg.end[e] = end;
        seg.tiles[e] = carry + sum - own;
        if (e == E - 1) {
          seg.start[E] = t;
          seg.tiles[E] = carry + sum;
        }
      }
      carry += __shfl_sync(0xffffffffu, sum, 31);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();   // both CTAs' barriers exist before anything signals them
  tc_fence_after();
  const uint32_t tmem = tmem_sh;
  Walk w(blockIdx.x >> 1);
  const int half = p.tn / 2;

  if (warp == 0) {
    if (lane == 0) {
      tma_prefetch_desc(&tm.w);
      tma_prefetch_desc(&tm.x);
      uint32_t it = 0;
      bool ok = true;
      while (ok && w.next(p, seg)) {
        const int row_w = w.e * p.n + w.f * FT + (int)rank * 128;
        const int row_x = w.r0 + (int)rank * (w.width() / 2);
        for (int k = 0; k < w.kn; k += HALVES, ++it) {
          const int st = it % STAGES;
          if (it >= STAGES && !mbar_wait_each(&empty[st], (it / STAGES - 1) & 1, p.err)) {
            ok = false;
            break;
          }
          uint8_t* dst = sm + st * STAGE_BYTES;
          const uint32_t bar = smem_cluster_addr(&full[st], 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[st], 2 * HALVES * (W_BYTES + half * KS));
#pragma unroll
          for (int h = 0; h < HALVES; ++h) {   // (a step behind the last one is zeros)
            tma_load_2d_pair(dst + h * W_BYTES, &tm.w, bar, (w.k0 + k + h) * KS, row_w);
            tma_load_2d_pair(dst + X_OFF + h * X_BYTES, &tm.x, bar, (w.k0 + k + h) * KS, row_x);
          }
        }
      }
      if (rank == 0) wait_landed(full, it, p.err);
    }
  } else if (warp == 1) {
    if (lane == 0 && rank == 0) {
      // This thread's own instructions are a good part of the pace (an MMA takes 112
      // clocks at the nominal rate): what can be is carried along, not computed.
      uint32_t group = 0, set = 0, tile = 0;
      uint32_t st = 0, parity = 0;         // the next stage and its phase
      bool ok = true;
      const uint32_t ring = sdesc_lo(smem_u32(sm), 16);
      uint32_t alo = ring;
      uint32_t d = 0;
      auto next_accumulator = [&] {
        const int buf = tile & 1;
        if (tile >= 2 && !mbar_wait_cluster(&acc_empty[buf], ((tile >> 1) - 1) & 1, p.err))
          return false;
        tc_fence_after();
        d = tmem + (uint32_t)(buf * TN_MAX);
        return true;
      };
      while (ok && w.next(p, seg)) {
        if (!CHAINS && !next_accumulator()) break;
        const int n = w.width();
        const bool wide = n > 128;
        const uint32_t idesc0 = idesc_mx(n, 0);
        uint32_t more = 0;
        for (int left = w.kn; ok && left > 0; left -= SF_STEPS, ++group) {
          if (CHAINS) {
            if (!next_accumulator()) {
              ok = false;
              break;
            }
            more = 0;
          }
          const int slot = group % SF_SLOTS;
          if (!mbar_wait_cluster(&sf_full[slot], (group / SF_SLOTS) & 1, p.err)) {
            ok = false;
            break;
          }
          tc_fence_after();
          uint32_t src = smem_u32(sm + SF_OFF + slot * (SF_WORDS * SF_BYTES));
          const int words = min(left, SF_STEPS);
          for (int i0 = 0; ok && i0 < words; i0 += 4, src += SF_BYTES) {
            const uint32_t sf = tmem + SF_COL + (uint32_t)(set++ % SF_SETS * SF_COLS);
            copy_scales_pair(sf, src);
            copy_scales_pair(sf + 4, src + 512);
            if (wide) copy_scales_pair(sf + 8, src + 1024);
            const int m = min(4, words - i0);
            uint32_t idesc = idesc0;
            for (int i = 0; i < m; i += HALVES) {
              if (!mbar_wait_each(&full[st], parity, p.err)) {
                ok = false;
                break;
              }
              tc_fence_after();
              const uint32_t now = st, a = alo, b = alo + (X_OFF >> 4);
              st = st + 1 == STAGES ? 0 : st + 1;
              parity ^= st == 0;
              alo = st == 0 ? ring : alo + (STAGE_BYTES >> 4);
#pragma unroll
              for (int h = 0; h < HALVES; ++h) {
                if (h > 0 && i + h >= m) break;
#pragma unroll
                for (int kk = 0; kk < KS / 32; ++kk)
                  mma_mx_pair(d, sdesc_make(a + (h * W_BYTES + kk * 32 >> 4)),
                              sdesc_make(b + (h * X_BYTES + kk * 32 >> 4)), idesc, sf, sf + 4,
                              h + kk > 0 ? 1u : more);
                idesc += 1u << 4 | 1u << 29;
              }
              more = 1;
              mma_commit_pair(&empty[now]);
            }
          }
          mma_commit_pair(&sf_empty[slot]);
          if (CHAINS) mma_commit_pair(&acc_full[tile++ & 1]);
        }
        if (!CHAINS) mma_commit_pair(&acc_full[tile++ & 1]);
      }
      // the MMAs are done before the pair's shared memory and TMEM are left
      if (tile > 0) mbar_wait_each(&acc_full[(tile - 1) & 1], ((tile - 1) >> 1) & 1, p.err);
    }
  } else if (warp == 2) {
    // Lane l holds the words of rows l, l + 32, ... of each 128.  A lane whose
    // wait gave up goes on without waiting and without telling anyone.
    uint32_t group = 0;
    uint32_t polls = kWaitPolls;
    while (w.next(p, seg)) {
      const int rows_b = max(p.experts, 1) * p.n;   // at most 2^24
      const int row_w = w.e * p.n + w.f * FT + (int)rank * 128;
      for (int k = 0; k < w.kn; k += SF_STEPS, ++group) {
        // k0 is a multiple of 4 steps: whole words of scale bytes
        const uint32_t off = (uint32_t)(p.cols + w.k0 + k);
        uint32_t v[SF_WORDS][12];
#pragma unroll
        for (int i = 0; i < 12; ++i) {
          const long long r = i < 4 ? row_w + 32 * i + lane : w.r0 + 32 * (i - 4) + lane;
          const bool in = i < 4 ? r < rows_b : r < w.r1;
          const uint8_t* src = (i < 4 ? p.b : p.a) + r * p.pitch + off;
#pragma unroll
          for (int j = 0; j < SF_WORDS; ++j)
            v[j][i] = in && k + 4 * j < w.kn ? *reinterpret_cast<const uint32_t*>(src + 4 * j) : 0u;
        }
        const int slot = group % SF_SLOTS;
        if (group >= SF_SLOTS)
          mbar_wait_or_pass(&sf_empty[slot], (group / SF_SLOTS - 1) & 1, polls, p.err);
        uint4* dst = reinterpret_cast<uint4*>(sm + SF_OFF + slot * (SF_WORDS * SF_BYTES)) + lane;
#pragma unroll
        for (int j = 0; j < SF_WORDS; ++j)
#pragma unroll
          for (int i = 0; i < 3; ++i)
            dst[j * (SF_BYTES / 16) + 32 * i] =
                make_uint4(v[j][4 * i], v[j][4 * i + 1], v[j][4 * i + 2], v[j][4 * i + 3]);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && polls) mbar_arrive_cluster(smem_cluster_addr(&sf_full[slot], 0));
      }
    }
  } else if (warp >= 4) {
    const int q = warp & 3;
    uint32_t polls = kWaitPolls;
    uint8_t* slot = sm + Ring<TN>::OUT_OFF + (warp - 4) * SLOT_BYTES;
    const int first = (warp - 4) / 4 * 32;
    if (lane == 0) tma_prefetch_desc(&tm.y);
    uint32_t tile = 0;
    uint32_t acc = 0;
    auto full_accumulator = [&] {
      mbar_wait_or_pass(&acc_full[tile & 1], (tile >> 1) & 1, polls, p.err);
      tc_fence_after();
      acc = tmem + (uint32_t)((tile & 1) * TN_MAX);
    };
    auto release_accumulator = [&] {
      tc_fence_before();
      __syncwarp();
      if (lane == 0 && polls) mbar_arrive_cluster(smem_cluster_addr(&acc_empty[tile & 1], 0));
      ++tile;
    };
    while (w.next(p, seg)) {
      const int col0 = w.f * FT + (int)rank * 128 + q * 32, n = w.r1 - w.r0;
      if constexpr (CHAINS) {
        // The tensor core drops what does not fit below the accumulator's last
        // place: sums of 7168 positive terms came out 1.1e-6 short, of 16384
        // 3.9e-6; as chains of 2048 that are added here, 3.7e-7 and 5.1e-7
        // (16384 x 7168 x 1536: 142 us, 134 us in one chain).
        constexpr int PARTS = (TN + 63) / 64;
        float v[PARTS][32];
        for (int k = 0; k < w.kn; k += SF_STEPS) {
          full_accumulator();
#pragma unroll
          for (int i = 0; i < PARTS; ++i) {
            if (first + 64 * i >= n) break;
            if (k == 0) {
              load_rows(tmem_addr(acc, q, first + 64 * i), v[i]);
            } else {
              float more[32];
              load_rows(tmem_addr(acc, q, first + 64 * i), more);
#pragma unroll
              for (int c = 0; c < 32; ++c) v[i][c] += more[c];
            }
          }
          release_accumulator();
        }
#pragma unroll
        for (int i = 0; i < PARTS; ++i) {
          if (first + 64 * i >= n) break;
          store_rows<float>(p, &tm.y, w, v[i], lane, first + 64 * i, col0, slot);
        }
        if (first == 0) store_zeros<float>(p, w, col0 + lane);
      } else {
        full_accumulator();
        for (int c0 = first; c0 < n; c0 += 64) {
          float v[32];
          load_rows(tmem_addr(acc, q, c0), v);
          if (p.bf16)
            store_rows<__nv_bfloat16>(p, &tm.y, w, v, lane, c0, col0, slot);
          else
            store_rows<float>(p, &tm.y, w, v, lane, c0, col0, slot);
        }
        release_accumulator();
        if (first == 0) {
          if (p.bf16)
            store_zeros<__nv_bfloat16>(p, w, col0 + lane);
          else
            store_zeros<float>(p, w, col0 + lane);
        }
      }
    }
    if (lane == 0) bulk_wait_read0();
    __syncwarp();
  }
  // neither CTA leaves while the pair's MMAs or the other CTA's arrivals may
  // still touch its shared memory or TMEM
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, TMEM_COLS);
  }
  cluster_sync();
}

// The pieces of K added up in order.
template <typename T>
__global__ void __launch_bounds__(256)
    mm8_join_kernel(const float* __restrict__ part, T* __restrict__ y, const int* __restrict__ end,
                    int rows, int n, int splits) {
  const long long all = (long long)rows * n;
  const long long used = (end ? (long long)min(rows, *end) : rows) * n;
  for (long long i = blockIdx.x * 256LL + threadIdx.x; i < used; i += gridDim.x * 256LL) {
    float s = part[i];
    for (int z = 1; z < splits; ++z) s += part[z * all + i];
    y[i] = from_f32<T>(s);
  }
}

// ---------------------------------------------------------------- host side
struct Mm8Plan {
  int tn, f_tiles, steps, splits, split_steps;
};

Mm8Plan mm8_plan(int rows, int K, int N, int experts) {
  Mm8Plan pl{};
  pl.f_tiles = (N + FT - 1) / FT;
  pl.steps = ck_cols(K) / KS;
  // Rows of a tile: the fewest clocks of the fullest pair, a step costing its
  // MMAs, or the bytes that it loads at about 45 a clock, or its issue.
  const int used = experts ? std::min(experts, rows) : 1;
  const int each = (rows + used - 1) / used;
  double best = -1.0;
  for (int tn = 32; tn <= TN_MAX; tn += 32) {
    const long long tiles = (long long)used * ((each + tn - 1) / tn) * pl.f_tiles;
    const long long turns = (tiles + PAIRS - 1) / PAIRS;
    const double step = std::max({2.0 * tn, (W_BYTES + tn / 2 * KS) / 45.0, 220.0});
    const double cost = turns * (pl.steps * step + 600.0);
    if (best < 0 || cost < best) {
      best = cost;
      pl.tn = tn;
    }
  }
  const long long tiles = (long long)used * ((each + pl.tn - 1) / pl.tn) * pl.f_tiles;
  // Pieces of K where the tiles leave half of the pairs without work: whole
  // words of scale bytes, 4 steps, at least
  const int words = (pl.steps + 3) / 4;
  int splits = 1;
  if (2 * tiles <= PAIRS) splits = (int)std::min<long long>(PAIRS / tiles, words);
  pl.split_steps = (words + splits - 1) / splits * 4;
  pl.splits = (pl.steps + pl.split_steps - 1) / pl.split_steps;
  return pl;
}

cudaError_t code_map(CUtensorMap* out, const void* base, uint64_t width, uint64_t rows,
                     uint64_t pitch, uint32_t box_rows) {
  auto enc = tmap_encoder();
  if (!enc) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {width, rows}, str[1] = {pitch};
  const cuuint32_t box[2] = {KS, box_rows}, one[2] = {1, 1};
  const CUresult r = enc(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, str,
                         box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                         CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// y (or the partial sums) [rows, n] in boxes of 32 columns x a slot's rows.
cudaError_t out_map(CUtensorMap* out, void* base, uint64_t n, uint64_t rows, bool bf16) {
  auto enc = tmap_encoder();
  if (!enc) return cudaErrorNotSupported;
  const uint32_t size = bf16 ? 2 : 4;
  const cuuint64_t dims[2] = {n, rows}, str[1] = {n * size};
  const cuuint32_t box[2] = {32, SLOT_BYTES / (32 * size)}, one[2] = {1, 1};
  const CUresult r =
      enc(out, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, base,
          dims, str, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE,
          CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

}  // namespace

size_t mm8_ws_bytes(int rows, int K, int N, int experts) {
  if (rows == 0) return 0;
  const Mm8Plan pl = mm8_plan(rows, K, N, experts);
  return pl.splits > 1 ? (size_t)pl.splits * rows * N * 4 : 0;
}

cudaError_t launch_mm8(int rows, int K, int N, int experts, bool fp32, const void* a,
                       const void* b, const int* start, const int* pair, void* y,
                       unsigned char* ws, int* err, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  const Mm8Plan pl = mm8_plan(rows, K, N, experts);
  Params p{};
  p.rows = rows; p.n = N; p.experts = experts;
  p.tn = pl.tn; p.f_tiles = pl.f_tiles; p.steps = pl.steps;
  p.splits = pl.splits; p.split_steps = pl.split_steps;
  p.pitch = ck_pitch(K); p.cols = ck_cols(K);
  p.bf16 = !fp32 && pl.splits == 1;
  p.a = static_cast<const uint8_t*>(a);
  p.b = static_cast<const uint8_t*>(b);
  p.start = start;
  p.pair = experts ? pair : nullptr;
  p.y = pl.splits > 1 ? static_cast<void*>(ws) : y;
  p.err = err;
  const int blocks = std::max(experts, 1);
  Maps tm;
  cudaError_t e;
  if ((e = code_map(&tm.w, b, p.cols, (uint64_t)blocks * N, p.pitch, 128)) != cudaSuccess) return e;
  if ((e = code_map(&tm.x, a, p.cols, rows, p.pitch, pl.tn / 2)) != cudaSuccess) return e;
  // rows that start on 16 bytes, and row numbers within a coordinate's 31 bits
  p.mapped = (uint64_t)N * (p.bf16 ? 2 : 4) % 16 == 0 && (long long)pl.splits * rows <= 0x7fffffff;
  tm.y = tm.x;
  if (p.mapped &&
      (e = out_map(&tm.y, p.y, N, (uint64_t)pl.splits * rows, p.bf16)) != cudaSuccess)
    return e;
  auto k = pl.tn > 32 ? fp32 ? mm8_kernel<TN_MAX, true> : mm8_kernel<TN_MAX, false>
                      : fp32 ? mm8_kernel<32, true> : mm8_kernel<32, false>;
  const int smem = pl.tn > 32 ? Ring<TN_MAX>::SMEM_BYTES : Ring<32>::SMEM_BYTES;
  if ((e = allow_smem(k, smem)) != cudaSuccess) return e;
  const long long most =
      ((long long)rows / pl.tn + std::min(blocks, rows)) * pl.f_tiles * pl.splits;
  {
    LaunchScope ls_("mm8", st);
    k<<<2 * (int)std::min<long long>(PAIRS, most), THREADS, smem, st>>>(tm, p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
  }
  if (pl.splits > 1) {
    const int grid = (int)std::min<long long>(((long long)rows * N + 255) / 256, 152 * 8);
    const int* end = experts ? start + experts : nullptr;
    LaunchScope ls_("mm8_join", st);
    const float* part = reinterpret_cast<const float*>(ws);
    if (fp32)
      mm8_join_kernel<<<grid, 256, 0, st>>>(part, static_cast<float*>(y), end, rows, N, pl.splits);
    else
      mm8_join_kernel<<<grid, 256, 0, st>>>(part, static_cast<__nv_bfloat16*>(y), end, rows, N,
                                            pl.splits);
  }
  return cudaGetLastError();
}

}  // namespace laga
