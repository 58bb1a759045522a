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

// end: device address of the number of rows, or null: all of them.
cudaError_t launch_ckpt_pack(int rows, int d, bool fp32, const void* x, const int* end, void* ck,
                             cudaStream_t st);
cudaError_t launch_ckpt_unpack(int rows, int d, bool fp32, const void* ck, void* x,
                               cudaStream_t st);

// Whether the sizes stay inside the kernel's 32-bit step counts.
bool ckpt_dw_fits(int rows, int d, int n, bool fp32);
size_t ckpt_dw_ws_bytes(int rows, int d, int n, bool fp32);
cudaError_t launch_ckpt_dw(int rows, int d, int n, bool fp32, const void* ck, const void* dy,
                           const float* gamma, float* dw, unsigned char* ws, int* err,
                           cudaStream_t st);

// ---- routing and experts
constexpr int ROUTE_MAX_EXPERTS = 1024, ROUTE_MAX_K = 32;
constexpr int ROUTE_ROW_NAN = -2;   // `row` of a NaN token's choice that found no expert

laga_status route_check(const laga_route_dims* dims);
long long route_rows(const laga_route_dims& d);
size_t route_ws_bytes(const laga_route_dims& d);
cudaError_t launch_route_fwd(const laga_route_dims& d, const void* logits, const float* bias,
                             int* expert, float* weight, int* row, int* pair, int* start,
                             unsigned char* ws, cudaStream_t st);
cudaError_t launch_route_bwd(const laga_route_dims& d, const void* logits, const int* expert,
                             const float* dweight, void* dlogits, cudaStream_t st);

// `end`: device address of the number of rows in use (start[experts]).
cudaError_t launch_spread8(int rows, int tokens, int top_k, int d, const void* ck, const int* pair,
                           const int* end, void* out, cudaStream_t st);
cudaError_t launch_combine_fwd(int tokens, int top_k, int rows, int d, bool fp32, const void* y,
                               const float* weight, const int* row, void* out, cudaStream_t st);
cudaError_t launch_combine_bwd(int tokens, int top_k, int rows, int d, bool fp32, const void* dout,
                               const void* y, const float* weight, const int* row, const int* pair,
                               const int* end, void* dy, float* dweight, cudaStream_t st);
cudaError_t launch_swiglu_fwd(int rows, int f, bool fp32, const void* gu, const int* end, void* ck,
                              cudaStream_t st);
cudaError_t launch_swiglu_bwd(int rows, int f, bool fp32, const void* gu, const void* da,
                              const int* end, void* dgu, cudaStream_t st);

cudaError_t launch_weight_pack(int experts, int K, int N, bool fp32, const void* w, void* fwd,
                               void* bwd, cudaStream_t st);
size_t mm8_ws_bytes(int rows, int K, int N, int experts);
cudaError_t launch_mm8(int rows, int K, int N, int experts, bool fp32, const void* a,
                       const void* b, const int* start, const int* pair, void* y,
                       unsigned char* ws, int* err, cudaStream_t st);

// Weight gradient by expert: the rows of expert e are start[e] .. start[e + 1],
// multiples of 128.
bool experts_dw_fits(int rows, int d, int n, int experts, bool fp32);
size_t experts_dw_ws_bytes(int rows, int d, int n, int experts, bool fp32);
cudaError_t launch_experts_dw(int rows, int d, int n, int experts, bool fp32, const void* ck,
                              const void* dy, const float* gamma, const int* start, float* dw,
                              unsigned char* ws, int* err, cudaStream_t st);

}  // namespace laga
