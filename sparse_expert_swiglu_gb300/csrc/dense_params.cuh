// Parameter blocks and launchers of the kernels on uncompressed weights.
#pragma once

#include <atomic>

#include "layer_plan.h"
#include "params.cuh"

namespace sesg {

struct LinearCall {
  int M, N, K;
  int bf16;             // x, w, bias, residual (and y unless out_f32): bf16, else fp16
  int kn;               // w is [K][N], else [N][K]
  int act;              // MOE_ACT_*
  int out_f32;
  int split;            // y as two rows for each token, the rounded value and what the rounding left
  int pairs;            // x has two such rows for each token of y: M = 2 tokens (no bias, act, w_mul)
  const void *x, *w, *w_mul, *bias, *bias_mul, *residual;
  void* y;
  size_t w_stride, w_mul_stride;  // elements between rows
  uint32_t tries;       // diagnostics (else 0): waits of so many rounds, of which the first CTA's run out
};

size_t linear_ws_bytes();
// Lets a kernel have all of an SM's shared memory; `done` keeps the devices (the first 64) that know it.
template <typename Kernel>
cudaError_t allow_shared(Kernel* kernel, std::atomic<uint64_t>& done, int smem_optin) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && done.load(std::memory_order_acquire) >> dev & 1)) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_optin);
  if (e == cudaSuccess && dev < 64) done.fetch_or(1ull << dev, std::memory_order_release);
  return e;
}

cudaError_t launch_linear(const LinearCall& c, void* ws, int sms, int smem_optin, cudaStream_t st);

struct DenseExpertSet {
  int E;
  const void *gate_t, *up_t, *down;  // [E][f][d]
  size_t gate_rs, up_rs, down_rs;    // elements between rows
};

struct DenseLayerCall {
  int B, d, f, k, renorm, rmsnorm, bf16;
  DenseExpertSet routed, shared;
  const void *x, *w_router, *residual;
  void* y;
  int32_t* user_idx;                 // optional copies of the routing
  float* user_w;
  uint32_t tries;                    // diagnostics (else 0): waits of so many rounds, ...
  int missing;                       // ... and the barrier over the grid that misses an arrival
};

size_t dense_layer_ws_bytes(int B, int d, int f, int E, int k, int ns, int sms);
cudaError_t launch_dense_layer(const DenseLayerCall& c, void* ws, int sms, int smem_optin, cudaStream_t st);

}  // namespace sesg
