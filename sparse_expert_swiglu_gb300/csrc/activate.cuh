// The products' activations (linear.cu, linear_int8.cu).
#pragma once

#include "common.cuh"

namespace sesg {

// One decision for W values, not one for each.  (silu_f's fast exponential is off by up to 2 + 1.2 |v| units in the last
// place: below the sums' own error where the result is not small beside |v|.)
// FAST: SiLU with the fast division too (2 units), for kernels that have 2000 of them to a tile: a precise one costs an SM a
// clock for every six values.  (Of v below -87.3 it gives 0, for -1e-36 and nearer to 0.)
template <int W, bool FAST = false>
__device__ __forceinline__ void activate(float (&v)[W], int act) {
  switch (act) {
    case MOE_ACT_RELU:
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];  // NaN stays NaN
      break;
    case MOE_ACT_GELU:
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] = 0.5f * v[i] * (1.f + erff(v[i] * 0.70710678118654752f));
      break;
    case MOE_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < W; ++i)
        v[i] = 0.5f * v[i] * (1.f + tanhf(0.79788456080286536f * (v[i] + 0.044715f * v[i] * v[i] * v[i])));
      break;
    case MOE_ACT_SILU:
#pragma unroll
      for (int i = 0; i < W; ++i) v[i] = FAST ? __fdividef(v[i], 1.f + __expf(-v[i])) : silu_f(v[i]);
      break;
    default: break;
  }
}

}  // namespace sesg
