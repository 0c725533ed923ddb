// The norms behind and before a block with its gate, its scale and the residual's:
//   s = residual_scale * residual + block_scale * gate (.) post(x),  y = norm(s), in 16 bits or 8-bit integers.
//
// Bound by HBM (with few tokens by the latency of its barriers): x and the residual are read once, a CTA keeps a token's
// row in registers in fp32 through both norms and writes s and y.  Variances are sums of squared differences from the mean, of
// values in registers.  With many tokens (norm_plan) a CTA goes from token to token, and while it works on one, every
// thread's own parts of the next come into shared memory by asynchronous copies.  Sums are formed in one order whatever the
// number of tokens: vectors of 8, then 32 neighbouring vectors as a tree, then those sums as a tree.
//
// Measured: 8192 tokens of 4096, two LayerNorms and an fp32 residual, 69 us (403 MB, 5.8 TB/s), with weights, biases and gates
// 72; RMSNorms and 8-bit tokens 57 us (235 MB; the conversions and the rounding bound it); one token 1.6 us, 64 of 6144 to 8 bits
// 3.9 us: launch, one latency of memory, a barrier for each sum.
#include "dense_params.cuh"
#include "int8.cuh"
#include "int8_params.cuh"
#include "norm_plan.h"

#include <cuda_bf16.h>

namespace sesg {

namespace {

struct NormArgs {
  // (bf16 and s_f32 choose the kernel on the host.  Without them here the compiler gives the kernels other registers: 8192 x 4096,
  // LayerNorms, 72 us for 68, 64 x 8192 3.04 for 2.91.)
  int M, d, bf16, s_f32, y_int8, post, norm, gate_every;
  int sectors;  // s starts on 32 bytes: whole sectors of fp32 at a time
  float residual_scale, block_scale, eps, per;  // per: 1 / d
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

// Sums of 32 neighbouring vectors, one of each lane, or of two such groups at once: lanes from 16 on have the second.  What a
// lane adds are the same two numbers at every step, whatever NV is.
template <int NV>
__device__ __forceinline__ float warp_sums(const float (&t)[NV], int lane) {
  // (with two, a lane keeps one and gives the other half's lanes what they add to theirs)
  const bool high = NV == 2 && (lane & 16);
  const float keep = high ? t[NV - 1] : t[0], give = NV == 1 ? keep : high ? t[0] : t[NV - 1];
  float v = keep + __shfl_xor_sync(0xffffffffu, give, 16);
#pragma unroll
  for (int o = 8; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The sum over the CTA of the vectors' sums, the same bits in all threads and for every NV; part: one of two arrays, by turns.
template <int NV>
__device__ __forceinline__ float block_sum(const float (&t)[NV], float* part) {
  const int warps = blockDim.x >> 5, lane = threadIdx.x & 31;
  float v = warp_sums<NV>(t, lane);
  if (lane % (32 / NV) == 0) part[(threadIdx.x >> 5) * NV + lane / (32 / NV)] = v;
  if (warps == 1) __syncwarp();
  else __syncthreads();
  const int groups = warps * NV;  // up to 64
  v = lane < groups ? part[lane] : 0.f;
  if (lane + 32 < groups) v += part[lane + 32];
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

__device__ __forceinline__ void copy16(void* to, const void* from) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(to)), "l"(from) : "memory");
}

// One token for each CTA at a time, NV vectors of 8 elements for each thread: a warp has 32 NV neighbouring ones, its lanes
// every 32nd.  AHEAD: the next token's come ahead.  BF16, S32: the types, known to the compiler (else 5 to 15 % more: 8192 x
// 4096, RMSNorms to 8 bits 64 us for 57).  With 64 registers a thread an SM holds 1024 threads.
template <int NV, bool AHEAD, int BF16, bool S32>
__global__ void __launch_bounds__(1024) residual_norm_kernel(const NormArgs p) {
  __shared__ float part[2][64];
  extern __shared__ uint4 next[];  // AHEAD: [NV][x, residual, the residual's second half][thread]
  griddep_launch_dependents();
  griddep_wait();
  const int T = blockDim.x, tid = threadIdx.x, n = p.d / 8, lane = tid & 31;
  const int c0 = (tid >> 5) * 32 * NV + lane;  // this thread's first vector
  const int each = p.residual ? S32 ? 3 : 2 : 1;  // vectors of 16 bytes
  auto ask = [&](int token) {
    const size_t at = (size_t)token * n;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = c0 + 32 * j;
      if (token >= p.M || c >= n) break;
      uint4* to = next + j * each * T + tid;
      copy16(to, reinterpret_cast<const uint4*>(p.x) + at + c);
      const uint4* from = reinterpret_cast<const uint4*>(p.residual);
      if (p.residual && !S32) copy16(to + T, from + at + c);
    }
    if (S32 && p.residual) {
      // 32 bytes of a thread: a warp copies its 1024 in their order, whole sectors at a time
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int c = (tid & ~31) * 2 + h * 32 + lane, k = 2 * (c0 - lane + 32 * j) + h * 32 + lane;
          if (token < p.M && k < 2 * n) copy16(next + (3 * j + 1) * T + c, reinterpret_cast<const uint4*>(p.residual) + 2 * at + k);
        }
    }
  };
  if (AHEAD) ask(blockIdx.x);
  int turn = 0;  // of the arrays, over all tokens: between two uses of one all warps meet at a barrier of the other
  for (int token = blockIdx.x; token < p.M; token += gridDim.x) {
  const size_t row = token, at = row * n;
  float v[NV][8];
  auto sum = [&](const float (&t)[NV]) {
    turn ^= 1;
    return block_sum<NV>(t, part[turn]);
  };
  auto normed = [&](int kind, const void* weight, const void* bias) {
    // One vector a thread: its weight and bias are under way while the sums are formed (8192 x 4096 takes two vectors a thread
    // and has no registers for them: 97 us for 79 with all vectors).
    uint4 early[2];
    if constexpr (NV == 1) {
      if (weight && c0 < n) early[0] = reinterpret_cast<const uint4*>(weight)[c0];
      if (bias && c0 < n) early[1] = reinterpret_cast<const uint4*>(bias)[c0];
    }
    if (kind == MOE_NORM_LAYER) {
      float t[NV] = {};
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (c0 + 32 * j < n) {
#pragma unroll
          for (int i = 0; i < 8; ++i) t[j] += v[j][i];
        }
      const float mean = sum(t) * p.per;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] -= mean;
    }
    float t[NV] = {};
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (c0 + 32 * j < n) {
#pragma unroll
        for (int i = 0; i < 8; ++i) t[j] = fmaf(v[j][i], v[j][i], t[j]);
      }
    const float inv = rsqrtf(fmaf(sum(t), p.per, p.eps));
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const int c = c0 + 32 * j;
      if (c >= n) break;
      float w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] *= inv;
      if (weight) {
        unpack8(NV == 1 ? early[0] : reinterpret_cast<const uint4*>(weight)[c], BF16, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] *= w[i];
      }
      if (bias) {
        unpack8(NV == 1 ? early[1] : reinterpret_cast<const uint4*>(bias)[c], BF16, w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[j][i] += w[i];
      }
    }
  };

  // x and the residual are asked for together
  uint4 r[NV][2];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = c0 + 32 * j;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    if (AHEAD) continue;
    const uint4 t = c < n ? reinterpret_cast<const uint4*>(p.x)[at + c] : zero;
    if (p.residual) {
      const uint4* from = reinterpret_cast<const uint4*>(p.residual);
      r[j][0] = c < n ? from[S32 ? 2 * (at + c) : at + c] : zero;
      r[j][1] = c < n && S32 ? from[2 * (at + c) + 1] : zero;
    }
    unpack8(t, BF16, v[j]);
  }
  if (AHEAD) {
    // what a thread reads its own warp has copied: no barrier of the CTA
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const uint4 zero = make_uint4(0, 0, 0, 0);
      const bool on = c0 + 32 * j < n;
      const uint4* from = next + j * each * T + tid;
      unpack8(on ? from[0] : zero, BF16, v[j]);
      if (p.residual) {
        r[j][0] = on ? S32 ? next[(3 * j + 1) * T + 2 * tid] : from[T] : zero;
        r[j][1] = on && S32 ? next[(3 * j + 1) * T + 2 * tid + 1] : zero;
      }
    }
    __syncwarp();
    ask(token + gridDim.x);
  }
  if (p.post) normed(p.post, p.post_weight, p.post_bias);
  const size_t gate_at = p.gate ? (size_t)((unsigned)token / (unsigned)p.gate_every) * n : 0;
  const uint4* gates = reinterpret_cast<const uint4*>(p.gate) + gate_at;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int c = c0 + 32 * j;
    if (c >= n) break;
    float w[8];
    if (p.gate) {
      unpack8(gates[c], BF16, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] *= w[i];
    }
    if (p.block_scale != 1.f) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] *= p.block_scale;
    }
    if (p.residual) {
      if (S32) unpack8(r[j][0], r[j][1], w);
      else unpack8(r[j][0], BF16, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = fmaf(p.residual_scale, w[i], v[j][i]);
    }
    if (p.s) {
      if (S32) {
        float* s = reinterpret_cast<float*>(p.s) + 8 * (at + c);
        if (p.sectors) {
          asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(s), "f"(v[j][0]), "f"(v[j][1]),
                       "f"(v[j][2]), "f"(v[j][3]), "f"(v[j][4]), "f"(v[j][5]), "f"(v[j][6]), "f"(v[j][7])
                       : "memory");
        } else {
          reinterpret_cast<float4*>(s)[0] = make_float4(v[j][0], v[j][1], v[j][2], v[j][3]);
          reinterpret_cast<float4*>(s)[1] = make_float4(v[j][4], v[j][5], v[j][6], v[j][7]);
        }
      } else {
        reinterpret_cast<uint4*>(p.s)[at + c] = pack8(v[j], BF16);
      }
    }
  }
  if (!p.norm) continue;
  normed(p.norm, p.weight, p.bias);
  if (!p.y_int8) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
      if (c0 + 32 * j < n) reinterpret_cast<uint4*>(p.y)[at + c0 + 32 * j] = pack8(v[j], BF16);
    continue;
  }
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (c0 + 32 * j < n) {
#pragma unroll
      for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[j][i]) & 0x7fffffffu);
    }
  m = warp_most(m);
  if (T > 32) {
    turn ^= 1;
    uint32_t* most = reinterpret_cast<uint32_t*>(part[turn]);
    if (lane == 0) most[tid >> 5] = m;
    __syncthreads();
    m = warp_most(lane < T / 32 ? most[lane] : 0);
  }
  const RowScale s = row_scale<false>(m);
  if (tid == 0) p.y_scale[row] = s.scale();
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (c0 + 32 * j < n) reinterpret_cast<uint2*>(p.y)[at + c0 + 32 * j] = quantize8<false>(v[j], s);
  }
}

}  // namespace

cudaError_t launch_residual_norm(const moe_residual_norm_t& op, int sms, cudaStream_t st) {
  NormArgs p;
  p.M = op.M;
  p.d = op.d;
  p.bf16 = op.dtype == MOE_BF16;
  p.s_f32 = op.s_dtype == MOE_F32;
  p.sectors = (uintptr_t)op.s % 32 == 0;
  p.y_int8 = op.y_dtype == MOE_I8;
  p.post = op.post;
  p.norm = op.norm;
  p.gate_every = op.gate ? op.M / op.gate_rows : 1;
  p.residual_scale = op.residual_scale;
  p.block_scale = op.block_scale;
  p.eps = op.eps;
  p.per = 1.f / op.d;
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
  const NormPlan l = norm_plan(op.M, op.d, op.residual != nullptr, p.s_f32, p.y_int8, sms);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(l.ctas);
  cfg.blockDim = dim3(l.threads);
  cfg.dynamicSmemBytes = l.bytes;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  using Kernel = void (*)(NormArgs);
  static constexpr Kernel kernels[4][3] = {
      {residual_norm_kernel<1, false, 0, false>, residual_norm_kernel<2, false, 0, false>, residual_norm_kernel<2, true, 0, false>},
      {residual_norm_kernel<1, false, 0, true>, residual_norm_kernel<2, false, 0, true>, residual_norm_kernel<2, true, 0, true>},
      {residual_norm_kernel<1, false, 1, false>, residual_norm_kernel<2, false, 1, false>, residual_norm_kernel<2, true, 1, false>},
      {residual_norm_kernel<1, false, 1, true>, residual_norm_kernel<2, false, 1, true>, residual_norm_kernel<2, true, 1, true>}};
  const int types = 2 * p.bf16 + p.s_f32;
  const Kernel kernel = kernels[types][l.ahead ? 2 : l.nv - 1];
  static std::atomic<uint64_t> allowed[4];
  if (l.ahead) {
    const cudaError_t e = allow_shared(kernel, allowed[types], kNormShared);
    if (e != cudaSuccess) return e;
  }
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace sesg
