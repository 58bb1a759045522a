// Host-side plans and launchers of the residual-stream operators and the
// 8-bit checkpoints (include/laga.h).  The plans make no CUDA call.
#pragma once

#include <cuda_runtime.h>

#include "../../include/laga.h"
#include "ckpt8.cuh"

namespace laga {

struct ResPtrs {
  const void *x = nullptr, *y = nullptr;        // forward inputs
  const void *dx_out = nullptr, *dh = nullptr;  // backward inputs
  const void *kept_y = nullptr, *kept_x = nullptr;
  const void* gate = nullptr;
  const float *alpha = nullptr, *gamma_post = nullptr, *gamma_pre = nullptr;
  float *stat_post = nullptr, *stat_pre = nullptr;
  void *x_out = nullptr, *h = nullptr, *ck_y = nullptr, *ck_x = nullptr;
  void *dx = nullptr, *dy = nullptr, *dgate = nullptr;
  float *dalpha = nullptr, *dgamma_post = nullptr, *dgamma_pre = nullptr;
  unsigned char* ws = nullptr;
  int* err = nullptr;
};

laga_status res_check(const laga_res_dims* dims);
size_t res_ws_bytes(const laga_res_dims& d);
cudaError_t launch_res_fwd(const laga_res_dims& d, const ResPtrs& x, cudaStream_t st);
cudaError_t launch_res_bwd(const laga_res_dims& d, const ResPtrs& x, cudaStream_t st);

cudaError_t launch_ckpt_pack(int rows, int d, bool fp32, const void* x, void* ck, cudaStream_t st);
cudaError_t launch_ckpt_unpack(int rows, int d, bool fp32, const void* ck, void* x,
                               cudaStream_t st);

// Whether the sizes stay inside the kernel's 32-bit step counts.
bool ckpt_dw_fits(int rows, int d, int n, bool fp32);
size_t ckpt_dw_ws_bytes(int rows, int d, int n, bool fp32);
cudaError_t launch_ckpt_dw(int rows, int d, int n, bool fp32, const void* ck, const void* dy,
                           const float* gamma, float* dw, unsigned char* ws, int* err,
                           cudaStream_t st);

}  // namespace laga
