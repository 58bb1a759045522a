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

// sigmoid(a) and 1 - sigmoid(a), each to fp32 accuracy (no cancellation)
LAGA_DEVINL float2 sigmoid_pair(float a) {
  const float e = expf(-fabsf(a));
  const float r = __fdividef(1.f, 1.f + e);
  return a >= 0.f ? make_float2(r, e * r) : make_float2(e * r, r);
}

// Launches of the ring kernels (residual_ring.cu); ring_ok says whether they
// take these dims, ring_slots how many column partials their backward writes.
bool ring_ok(const laga_res_dims& d, bool bwd);
int ring_slots(const laga_res_dims& d);
cudaError_t launch_ring_fwd(const laga_res_dims& d, const ResArgs& a, cudaStream_t st);
cudaError_t launch_ring_bwd(const laga_res_dims& d, const ResArgs& a, cudaStream_t st);

}  // namespace laga
