// Parameter blocks and launchers of the kernels on 8-bit integers and of the norms around a block.
#pragma once

#include "params.cuh"

namespace sesg {

cudaError_t launch_quantize(const void* x, int dtype, int rows, int K, int8_t* q, float* scale, cudaStream_t st);

struct LinearInt8Call {
  int M, N, K;
  int x16;              // x in 16 bits, quantised on the way; else int8 with x_scale
  int bf16, act, out_f32;
  const void* x;
  const float* x_scale;
  const int8_t *w, *w_mul;
  const float *w_scale, *w_mul_scale;
  const void *bias, *bias_mul, *residual;
  void* y;
};

cudaError_t launch_linear_int8(const LinearInt8Call& c, void* ws, int sms, int smem_optin, cudaStream_t st);

cudaError_t launch_residual_norm(const moe_residual_norm_t& op, cudaStream_t st);

}  // namespace sesg
