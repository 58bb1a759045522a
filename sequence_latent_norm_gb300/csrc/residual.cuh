// What the residual-stream kernels share (residual.cu: rows of any width;
// residual_ring.cu: rows of a multiple of 8 channels that fit its rings).
#pragma once

#include "ckpt8.cuh"
#include "common.cuh"
#include "kernels.h"
#include "ops.h"

namespace laga {

constexpr int kSms = 152;           // persistent CTAs of a launch are counted against this

struct ResArgs {
  int rows, d;
  int post, pre, norm_post, norm_pre, gate, ckpt;
  float eps, inv_d;
  ResPtrs x;
  float *part_post, *part_pre, *part_alpha;   // column partials [slots, d], [slots]
};

// sigmoid(a) = 1 / (1 + e^-a) and 1 - sigmoid(a) = e^-a sigmoid(a), without
// cancellation on either side.  e^-a is 2^t, t = -a log2 e, by the hardware's
// exponential (within 2^-22 of itself); the rounded product and constant move
// it by another 1.23 |a| 2^-24 of itself.  Both results stay within (1.25 |a|
// + 9) 2^-24 of themselves: far below a bf16 step, and for fp32 no more than
// the gate's own rounding (a half step of a moves e^-a by |a| 2^-24) and a few
// units.
//
// Below -87.3 the sigmoid would be subnormal: it is zero, so that a gate of
// -inf shuts (and 1 - sigmoid(a) is given as zero with it: it only ever
// multiplies sigmoid(a)).  a is held at -88.5 and above, where e^-a is finite.
LAGA_DEVINL float2 sigmoid_pair(float a) {
  float e, s;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(a) : "f"(a), "f"(-88.5f));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(a * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(s) : "f"(1.f + e));
  return make_float2(s, e * s);
}

// Launches of the ring kernels (residual_ring.cu); ring_ok says whether they
// take these dims, ring_slots how many column partials their backward writes.
bool ring_ok(const laga_res_dims& d, bool bwd);
int ring_slots(const laga_res_dims& d);
cudaError_t launch_ring_fwd(const laga_res_dims& d, const ResArgs& a, cudaStream_t st);
cudaError_t launch_ring_bwd(const laga_res_dims& d, const ResArgs& a, cudaStream_t st);

}  // namespace laga
