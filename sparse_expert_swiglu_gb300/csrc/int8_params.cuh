// Parameter blocks and launchers of the kernels on 8-bit integers and of the norms around a block.
#pragma once

#include "params.cuh"

namespace sesg {

cudaError_t launch_quantize(const void* x, int dtype, int rows, int K, int8_t* q, float* scale, int sms, cudaStream_t st);

// The tokens of the kernel that runs behind it (linear_int8_tiles.cu): fp16 integers [M][K], and scales with room for a
// multiple of 16.  dtype MOE_I8: x with its scales, else x is quantised.
cudaError_t launch_tokens(const void* x, int dtype, const float* x_scale, int M, int K, void* tokens, float* scales, int sms,
                          cudaStream_t st);

struct LinearInt8Call {
  int M, N, K;
  int x_dtype;          // MOE_I8 with x_scale; else MOE_F32 or the type in 16 bits, quantised on the way
  int bf16, act, out_f32;
  const void* x;
  const float* x_scale;
  const int8_t *w, *w_mul;
  const float *w_scale, *w_mul_scale;
  const void *bias, *bias_mul, *residual;
  void* y;
  uint32_t tries;       // diagnostics (else 0): waits of so many rounds, of which the first CTA's run out
};

// Workspace of a product: the head, then the tokens as fp16 integers and their scales.
struct Int8Ws {
  size_t tokens, scales, bytes;
  Int8Ws(int M, int K);
};

cudaError_t launch_linear_int8(const LinearInt8Call& c, void* ws, int sms, int smem_optin, cudaStream_t st);
cudaError_t launch_int8_tiles(const LinearInt8Call& c, const void* tokens, const float* scales, void* ws, int sms,
                              int smem_optin, cudaStream_t st);

cudaError_t launch_residual_norm(const moe_residual_norm_t& op, int sms, cudaStream_t st);

}  // namespace sesg
