// y = act(s_x s_w (x w^T) + bias) [* (s_x s_mul (x w_mul^T) + bias_mul)] [+ residual] on 8-bit integers.
//
// Few tokens: a stream of w, bound by HBM.  A warp takes RW neighbouring rows of w (with w_mul the same rows of both) at a
// time, 16 bytes a lane and load, the next loads in flight while it multiplies; the tokens lie in shared memory, where every
// CTA quantises them itself.  Four products and their sum are one instruction (dp4a: 254 products a clock and SM, of which
// HBM's rate needs 23 for each token); sums are integers, so that their order is free.  Rows at a time: with one token one row
// gives the most loads in flight, with more each token's read from shared memory serves RW rows (4 tokens of 4096 x 14336 with
// 2 rows 15.8 us, with 4 14.7).  Measured: 1 token of 32000 x 4096 25.5 us (5.1 TB/s; about 6 us of that are a call's own:
// launch 0.7, the token's two passes behind w's first loads 2.9, first products 1.1, an end), of 4096 x 4096 6.4 us.
#include "activate.cuh"
#include "dense.cuh"
#include "dense_params.cuh"
#include "int8.cuh"
#include "int8_params.cuh"

namespace sesg {

namespace {

constexpr int kFewThreads = 512, kFewWarps = kFewThreads / 32;
constexpr int kFewShared = 200 << 10;  // bytes of tokens

struct Int8Args {
  int M, N, K, bf16, act, out_f32;
  int x_dtype;          // MOE_I8, MOE_F32, else 16 bits
  int log_parts;        // warps that share a row along k: 2 to that power
  const void* x;
  const float* x_scale;
  const int8_t *w, *w_mul;
  const float *w_scale, *w_mul_scale;
  const void *bias, *bias_mul, *residual;
  void* y;
};

__device__ __forceinline__ void store_one(const Int8Args& p, int tok, int row, int sum, int sum_mul, float xs) {
  float v[1] = {int8_value(sum, xs, p.w_scale[row], p.bias ? ld16(p.bias, row, p.bf16) : 0.f)};
  activate<1, true>(v, p.act);
  if (p.w_mul)
    v[0] = __fmul_rn(v[0], int8_value(sum_mul, xs, p.w_mul_scale[row], p.bias_mul ? ld16(p.bias_mul, row, p.bf16) : 0.f));
  const size_t at = (size_t)tok * p.N + row;
  if (p.residual) v[0] = __fadd_rn(v[0], ld16(p.residual, at, p.bf16));
  if (p.out_f32) reinterpret_cast<float*>(p.y)[at] = v[0];
  else reinterpret_cast<unsigned short*>(p.y)[at] = to16(v[0], p.bf16);
}

// The nt tokens as integers in shared memory, and their scales.
__device__ __forceinline__ void few_tokens(const Int8Args& p, int nt, int8_t* xq, float* scales, uint32_t* most) {
  const int tid = threadIdx.x;
  if (p.x_dtype == MOE_I8) {
    const uint4* from = reinterpret_cast<const uint4*>(p.x);
    for (int i = tid; i < nt * (p.K / 16); i += kFewThreads) reinterpret_cast<uint4*>(xq)[i] = from[i];
    if (tid < nt) scales[tid] = p.x_scale[tid];
    __syncthreads();
    return;
  }
  const int n = p.K / 8;
  const bool f32 = p.x_dtype == MOE_F32;
  const uint4* from = reinterpret_cast<const uint4*>(p.x);
  if (tid < nt) most[tid] = 0;
  __syncthreads();
  for (int t = 0; t < nt; ++t) {
    uint32_t m = 0;
    if (f32) {
      for (int i = tid; i < 2 * n; i += kFewThreads) m = most32(m, from[(size_t)t * 2 * n + i]);
    } else {
      for (int i = tid; i < n; i += kFewThreads) m = most16(m, from[(size_t)t * n + i]);
      m = most_f32(m, p.bf16);
    }
    m = warp_most(m);
    if ((tid & 31) == 0) atomicMax(&most[t], m);
  }
  __syncthreads();
  for (int t = 0; t < nt; ++t) {
    const RowScale s = f32 ? row_scale<false>(most[t]) : row_scale<true>(most[t]);
    if (tid == 0) scales[t] = s.scale();
    for (int i = tid; i < n; i += kFewThreads) {
      float v[8];
      if (f32) unpack8(from[((size_t)t * n + i) * 2], from[((size_t)t * n + i) * 2 + 1], v);
      else unpack8(from[(size_t)t * n + i], p.bf16, v);
      reinterpret_cast<uint2*>(xq)[t * n + i] = f32 ? quantize8<false>(v, s) : quantize8<true>(v, s);
    }
  }
  __syncthreads();
}

// Up to TOK tokens; RW rows of w for a warp at a time.
template <int TOK, int RW>
__global__ void __launch_bounds__(kFewThreads, 1) int8_few_kernel(const Int8Args p) {
  constexpr int U = (TOK == 16 ? 4 : 8) / RW;  // loads of a row in flight
  extern __shared__ __align__(16) int8_t xq[];
  __shared__ float scales[TOK];
  __shared__ uint32_t most[TOK];
  __shared__ int shared_sums[2][2][kFewWarps][32];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int V = p.K / 16, segs = (V + 31) / 32, groups = (p.N + RW - 1) / RW;
  const int part = warp & ((1 << p.log_parts) - 1), team = warp >> p.log_parts, per = kFewWarps >> p.log_parts;
  const int s0 = segs * part >> p.log_parts, s1 = segs * (part + 1) >> p.log_parts;
  const int mats = p.w_mul ? 2 : 1;
  const int first = team * gridDim.x + blockIdx.x, step = per * gridDim.x;

  // a batch: U segments of 32 loads of the group's rows in one matrix
  struct At {
    int g, mat, s;
  };
  auto fetch = [&](const At& a, uint4 (&v)[RW][U]) {
    const uint4* base = reinterpret_cast<const uint4*>(a.mat ? p.w_mul : p.w);
#pragma unroll
    for (int r = 0; r < RW; ++r) {
      const int row = a.g * RW + r;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = (a.s + u) * 32 + lane;
        v[r][u] = row < p.N && a.s + u < s1 && i < V ? ld_stream_v4(base + (size_t)row * V + i) : make_uint4(0, 0, 0, 0);
      }
    }
  };
  uint4 cur[RW][U], next[RW][U];
  int acc[RW][TOK], kept = 0, round = 0;  // kept: this lane's sum of w, (row, token) = lane
  auto clear = [&] {
#pragma unroll
    for (int r = 0; r < RW; ++r)
#pragma unroll
      for (int t = 0; t < TOK; ++t) acc[r][t] = 0;
  };
  clear();
  const int nt = p.M;
  At a = {first, 0, s0};
  if (a.g < groups) fetch(a, cur);
  few_tokens(p, nt, xq, scales, most);
  while (a.g < groups) {
    At b = {a.g, a.mat, a.s + U};
    if (b.s >= s1) {
      b.s = s0;
      if (++b.mat == mats) {
        b.mat = 0;
        b.g += step;
      }
    }
    if (b.g < groups) fetch(b, next);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = (a.s + u) * 32 + lane, at = i < V ? i : 0;  // (behind the row: zeros times anything)
#pragma unroll
      for (int t = 0; t < TOK; ++t) {
        if (t < nt) {
          const uint4 x = reinterpret_cast<const uint4*>(xq)[(size_t)t * V + at];
#pragma unroll
          for (int r = 0; r < RW; ++r) {
            acc[r][t] = __dp4a((int)cur[r][u].x, (int)x.x, acc[r][t]);
            acc[r][t] = __dp4a((int)cur[r][u].y, (int)x.y, acc[r][t]);
            acc[r][t] = __dp4a((int)cur[r][u].z, (int)x.z, acc[r][t]);
            acc[r][t] = __dp4a((int)cur[r][u].w, (int)x.w, acc[r][t]);
          }
        }
      }
    }
    if (b.g != a.g || b.mat != a.mat) {  // the rows' end in this matrix
      int mine = 0;
#pragma unroll
      for (int r = 0; r < RW; ++r)
#pragma unroll
        for (int t = 0; t < TOK; ++t) {
          const int s = __reduce_add_sync(0xffffffffu, acc[r][t]);
          if (lane == r * TOK + t) mine = s;
        }
      clear();
      if (p.log_parts) shared_sums[round & 1][a.mat][warp][lane] = mine;
      if (b.g == a.g) {
        kept = mine;
      } else {
        int sum = mats == 2 ? kept : mine, sum_mul = mine;
        if (p.log_parts) {
          named_barrier(1 + team, 32 << p.log_parts);
          sum = sum_mul = 0;
          if (part == 0)
            for (int i = 0; i < 1 << p.log_parts; ++i) {
              sum += shared_sums[round & 1][0][warp + i][lane];
              sum_mul += shared_sums[round & 1][mats - 1][warp + i][lane];
            }
        }
        ++round;
        const int row = a.g * RW + lane / TOK, tok = lane % TOK;
        if (part == 0 && lane < RW * TOK && row < p.N && tok < nt) store_one(p, tok, row, sum, sum_mul, scales[tok]);
      }
    }
    a = b;
#pragma unroll
    for (int r = 0; r < RW; ++r)
#pragma unroll
      for (int u = 0; u < U; ++u) cur[r][u] = next[r][u];
  }
}

}  // namespace

Int8Ws::Int8Ws(int M, int K) {
  auto up = [](size_t v) { return (v + 255) / 256 * 256; };
  tokens = up(linear_ws_bytes());
  scales = tokens + up((size_t)M * K * 2);
  bytes = scales + up((size_t)M * 4 + 60);
}

// Whether the stream of w takes the call, and not the tensor cores.  The stream is a single short kernel (512 x 512: 2.8 us
// for 4 tokens and 4.3 for 16 against 5.3) whose time grows with tokens times weights, faster where there are more than 4 and
// more than 8 tokens.  They meet, in us of stream and tensor cores, for up to 4 tokens at about 450e6 of them (4 of 32000 x
// 4096 27.5 and 27.3, of 14336 x 4096 15.1 and 15.9), up to 8 at 280e6 (8 of 8192 x 4096 11.9 and 12.9, 6 of 4096 x 14336
// 16.5 both, 5 of 14336 x 4096 17.3 and 15.7), up to 16 at 70e6 (16 of 4096 x 1024 6.1 and 6.7, 9 of 2048 x 8192 10.7 both,
// 9 of 4096 x 4096 10.4 and 9.3, 16 12.8 and 9.4).
static bool int8_few(int M, int N, int K, bool gated, int tok) {
  const double work = (gated ? 2.0 : 1.0) * N * K * M;
  return M == 1 || (M <= tok && tok * K <= kFewShared && (M <= 2 || work <= (M <= 4 ? 450e6 : M <= 8 ? 280e6 : 70e6)));
}

cudaError_t launch_linear_int8(const LinearInt8Call& c, void* ws, int sms, int smem_optin, cudaStream_t st) {
  const int tok = c.M <= 1 ? 1 : c.M <= 2 ? 2 : c.M <= 4 ? 4 : c.M <= 8 ? 8 : 16;
  if (!int8_few(c.M, c.N, c.K, c.w_mul != nullptr, tok) || c.tries) {
    const Int8Ws at(c.M, c.K);
    uint8_t* base = reinterpret_cast<uint8_t*>(ws);
    float* scales = reinterpret_cast<float*>(base + at.scales);
    cudaError_t e = launch_tokens(c.x, c.x_dtype, c.x_scale, c.M, c.K, base + at.tokens, scales, sms, st);
    if (e == cudaSuccess) e = launch_int8_tiles(c, base + at.tokens, scales, ws, sms, smem_optin, st);
    return e;
  }
  Int8Args p;
  p.M = c.M;
  p.N = c.N;
  p.K = c.K;
  p.x_dtype = c.x_dtype;
  p.bf16 = c.bf16;
  p.act = c.act;
  p.out_f32 = c.out_f32;
  p.x = c.x;
  p.x_scale = c.x_scale;
  p.w = c.w;
  p.w_mul = c.w_mul;
  p.w_scale = c.w_scale;
  p.w_mul_scale = c.w_mul_scale;
  p.bias = c.bias;
  p.bias_mul = c.bias_mul;
  p.residual = c.residual;
  p.y = c.y;
  const int rw = tok == 1 ? 1 : tok == 4 || tok == 8 ? 4 : 2, groups = (c.N + rw - 1) / rw;
  const int segs = (c.K / 16 + 31) / 32;
  int parts = 1;
  for (p.log_parts = 0; parts < kFewWarps && parts * 2 <= segs && (long long)groups * parts * 2 <= (long long)sms * kFewWarps;
       ++p.log_parts)
    parts *= 2;
  using Kernel = void (*)(Int8Args);
  const Kernel kernel = tok == 1 ? int8_few_kernel<1, 1> : tok == 2 ? int8_few_kernel<2, 2>
                        : tok == 4 ? int8_few_kernel<4, 4> : tok == 8 ? int8_few_kernel<8, 4> : int8_few_kernel<16, 2>;
  static std::atomic<uint64_t> allowed[5];
  cudaError_t e = allow_shared(kernel, allowed[tok == 1 ? 0 : tok == 2 ? 1 : tok == 4 ? 2 : tok == 8 ? 3 : 4], kFewShared);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(groups < sms ? groups : sms);
  cfg.blockDim = dim3(kFewThreads);
  cfg.dynamicSmemBytes = (size_t)tok * c.K;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace sesg
