// The norms behind and before a block with its gate, its scale and the residual's:
//   s = residual_scale * residual + block_scale * gate (.) post(x),  y = norm(s), in 16 bits or 8-bit integers.
//
// Bound by HBM (with few tokens by the latency of its barriers): x and the residual are read once, a CTA for each token
// keeps the row in registers in fp32 through both norms and writes s and y.  Variances are sums of squared
// differences from the mean, of values in registers.
#include "int8.cuh"
#include "int8_params.cuh"

#include <cuda_bf16.h>

namespace sesg {

namespace {

struct NormArgs {
  int d, bf16, s_f32, y_int8, post, norm, gate_every;
  float residual_scale, block_scale, eps;
  const void *x, *residual, *gate, *post_weight, *post_bias, *weight, *bias;
  void *s, *y;
  float* y_scale;
};

__device__ __forceinline__ uint4 pack8(const float (&v)[8], int bf16) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (bf16) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    } else {
      const __half2 h = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A sum over the CTA's threads, the same bits in all of them; part: one of two arrays, used by turns.
__device__ __forceinline__ float block_sum(float v, float* part) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  if (warps == 1) return v;
  if (lane == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = lane < warps ? part[lane] : 0.f;
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// One token for each CTA, NV vectors of 8 elements for each thread.
template <int NV>
__global__ void __launch_bounds__(NV == 1 ? 1024 : 512) residual_norm_kernel(const NormArgs p) {
  __shared__ float part[2][32];
  griddep_launch_dependents();
  griddep_wait();
  const int T = blockDim.x, tid = threadIdx.x, n = p.d / 8;
  const size_t row = blockIdx.x, at = row * n;
  int turn = 0;
  float v[NV][8];
  auto sum = [&](float t) {
    turn ^= 1;
    return block_sum(t, part[turn]);
  };
  auto normed = [&](int kind, const void* weight, const void* bias) {
    if (kind == MOE_NORM_LAYER) {
      float t = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (tid + j * T < n) {
#pragma unroll
          for (int i = 0; i < 8; ++i) t += v[j][i];
        }
      const float mean = sum(t) / p.d;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] -= mean;
    }
    float t = 0.f;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (tid + j * T < n) {
#pragma unroll
        for (int i = 0; i < 8; ++i) t = fmaf(v[j][i], v[j][i], t);
      }
    const float inv = 1.f / sqrtf(sum(t) / p.d + p.eps);
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = tid + j * T;
      if (c >= n) break;
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] *= inv;
      if (weight) {
        unpack8(reinterpret_cast<const uint4*>(weight)[c], p.bf16, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] *= w[i];
      }
      if (bias) {
        unpack8(reinterpret_cast<const uint4*>(bias)[c], p.bf16, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] += w[i];
      }
    }
  };

#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = tid + j * T;
    const uint4 t = c < n ? reinterpret_cast<const uint4*>(p.x)[at + c] : make_uint4(0, 0, 0, 0);
    unpack8(t, p.bf16, v[j]);
  }
  if (p.post) normed(p.post, p.post_weight, p.post_bias);
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = tid + j * T;
    if (c >= n) break;
    float w[8];
    if (p.gate) {
      unpack8(reinterpret_cast<const uint4*>(p.gate)[row / p.gate_every * n + c], p.bf16, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] *= w[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) v[j][i] *= p.block_scale;
    if (p.residual) {
      if (p.s_f32) {
        const float4* r = reinterpret_cast<const float4*>(p.residual) + 2 * (at + c);
        const float4 a = r[0], b = r[1];
        const float t[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = t[i];
      } else {
        unpack8(reinterpret_cast<const uint4*>(p.residual)[at + c], p.bf16, w);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = fmaf(p.residual_scale, w[i], v[j][i]);
    }
    if (p.s) {
      if (p.s_f32) {
        float4* s = reinterpret_cast<float4*>(p.s) + 2 * (at + c);
        s[0] = make_float4(v[j][0], v[j][1], v[j][2], v[j][3]);
        s[1] = make_float4(v[j][4], v[j][5], v[j][6], v[j][7]);
      } else {
        reinterpret_cast<uint4*>(p.s)[at + c] = pack8(v[j], p.bf16);
      }
    }
  }
  if (!p.norm) return;
  normed(p.norm, p.weight, p.bias);
  if (!p.y_int8) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (tid + j * T < n) reinterpret_cast<uint4*>(p.y)[at + tid + j * T] = pack8(v[j], p.bf16);
    return;
  }
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (tid + j * T < n) {
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[j][i]) & 0x7fffffffu);
    }
  m = warp_most(m);
  if (T > 32) {
    uint32_t* most = reinterpret_cast<uint32_t*>(part[turn ^ 1]);
    if ((tid & 31) == 0) most[tid >> 5] = m;
    __syncthreads();
    m = warp_most((tid & 31) < T / 32 ? most[tid & 31] : 0);
  }
  const RowScale s = row_scale(m);
  if (tid == 0) p.y_scale[row] = s.scale;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (tid + j * T < n) reinterpret_cast<uint2*>(p.y)[at + tid + j * T] = quantize8(v[j], s);
}

}  // namespace

cudaError_t launch_residual_norm(const moe_residual_norm_t& op, cudaStream_t st) {
  NormArgs p;
  p.d = op.d;
  p.bf16 = op.dtype == MOE_BF16;
  p.s_f32 = op.s_dtype == MOE_F32;
  p.y_int8 = op.y_dtype == MOE_I8;
  p.post = op.post;
  p.norm = op.norm;
  p.gate_every = op.gate ? op.M / op.gate_rows : 1;
  p.residual_scale = op.residual_scale;
  p.block_scale = op.block_scale;
  p.eps = op.eps;
  p.x = op.x;
  p.residual = op.residual;
  p.gate = op.gate;
  p.post_weight = op.post_weight;
  p.post_bias = op.post_bias;
  p.weight = op.weight;
  p.bias = op.bias;
  p.s = op.s;
  p.y = op.y;
  p.y_scale = op.y_scale;
  const int n = op.d / 8, nv = n <= 512 ? 1 : n <= 1024 ? 2 : 4;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(op.M);
  cfg.blockDim = dim3(((n + nv - 1) / nv + 31) / 32 * 32);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const auto kernel = nv == 1 ? residual_norm_kernel<1> : nv == 2 ? residual_norm_kernel<2> : residual_norm_kernel<4>;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace sesg
