// What the residual-stream kernels share (residual.cu: rows of any width;
// residual_ring.cu: rows of a multiple of 8 channels).
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
// cancellation on either side.  e^-a is 2^(-a log2 e) by the hardware's
// exponential: the product's rounding leaves it within 0.7 |a| 2^-24 and 2 ulp
// of itself.  Below -87 the sigmoid stays at e^-87, the end of the normal
// range, so that e^-a is finite.
LAGA_DEVINL float2 sigmoid_pair(float a) {
  float e, s;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(a) : "f"(a), "f"(-87.f));
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
