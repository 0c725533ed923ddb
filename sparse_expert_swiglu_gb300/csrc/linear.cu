// y = act(x w^T + bias) [* (x w_mul^T + bias_mul)] [+ residual] on 16-bit x and w, fp32 sums.
//
// The features lie on the 128 TMEM lanes, the tokens on the columns: a tile is 256 features
// (two products of 128 that share the token operand; with w_mul 128 features of each matrix)
// by up to 256 tokens.  With few tokens the call is a stream of w, bound by HBM: the work is
// cut along k so that every SM streams an equal share, and the last share of a tile to come
// adds the others' partial sums (in the order of k) and runs the epilogue.  With many tokens
// it is bound by the tensor cores.
#include "dense.cuh"
#include "dense_params.cuh"

namespace sesg {

namespace {

struct LinearArgs {
  int M, N, MT, NT, gated, bf16, kn, act, out_f32;
  Sched s;
  const void *bias, *bias_mul, *residual;
  void* y;
  float* part;      // [segment][2][NT][128]
  DenseHead* head;
  int stages, acc_bufs, tmem_cols, stream;
};

// One decision for 16 values, not one for each.
__device__ __forceinline__ void activate(float (&v)[16], int act) {
  switch (act) {
    case MOE_ACT_RELU:
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = v[i] < 0.f ? 0.f : v[i];  // NaN stays NaN
      break;
    case MOE_ACT_GELU:
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0.5f * v[i] * (1.f + erff(v[i] * 0.70710678118654752f));
      break;
    case MOE_ACT_GELU_TANH:
#pragma unroll
      for (int i = 0; i < 16; ++i)
        v[i] = 0.5f * v[i] * (1.f + tanhf(0.79788456080286536f * (v[i] + 0.044715f * v[i] * v[i] * v[i])));
      break;
    case MOE_ACT_SILU:
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = silu_f(v[i]);
      break;
    default: break;
  }
}

// Residual and store of 16 tokens' values of one feature; token i at offset at + i * N.
template <bool FULL>
__device__ __forceinline__ void linear_write(const LinearArgs& p, size_t at, int n, float (&v)[16]) {
  if (p.residual) {
    const unsigned short* r = reinterpret_cast<const unsigned short*>(p.residual) + at;
    unsigned short t[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) t[i] = FULL || i < n ? r[(size_t)i * p.N] : (unsigned short)0;
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] += from16(t[i], p.bf16);
  }
  if (p.out_f32) {
    float* y = reinterpret_cast<float*>(p.y) + at;
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (FULL || i < n) y[(size_t)i * p.N] = v[i];
  } else {
    unsigned short* y = reinterpret_cast<unsigned short*>(p.y) + at;
    unsigned short t[16];
    if (p.bf16) {
#pragma unroll
      for (int i = 0; i < 16; ++i) t[i] = to16(v[i], 1);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) t[i] = to16(v[i], 0);
    }
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if (FULL || i < n) y[(size_t)i * p.N] = t[i];
  }
}

// Epilogue of 16 tokens of one feature: v, and with w_mul m, are the sums; n tokens from t0 exist.
__device__ __forceinline__ void linear_store(const LinearArgs& p, int feat, int t0, int n, float bias, float bias_mul,
                                             float (&v)[16], const float (&m)[16], bool gated) {
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] += bias;
  activate(v, p.act);
  if (gated) {
#pragma unroll
    for (int i = 0; i < 16; ++i) v[i] *= m[i] + bias_mul;
  }
  const size_t at = (size_t)t0 * p.N + feat;
  if (n >= 16) linear_write<true>(p, at, n, v);
  else linear_write<false>(p, at, n, v);
}

__global__ void __launch_bounds__(kDnThreads, 1)
linear_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mw2,
              const __grid_constant__ CUtensorMap mx, const LinearArgs p) {
  extern __shared__ uint8_t raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const uint32_t stage_bytes = kDnBytesA + p.NT * 128;
  DenseBars* bars = reinterpret_cast<DenseBars*>(ring + (size_t)p.stages * stage_bytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;
  const int S = p.stages, NT = p.NT;
  const int width = p.gated ? kDnHalf : 2 * kDnHalf;  // features of a tile
  int* status = &p.head->ctrl.status;
  volatile int* abort = &bars->abort;

  if (tid == 0) {
    dn_init_bars(bars);
    tma_prefetch_map(&mw);
    tma_prefetch_map(&mx);
    if (p.gated) tma_prefetch_map(&mw2);
  }
  if (warp == 2) tmem_alloc(&bars->tmem, p.tmem_cols);
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  const uint32_t tmem = bars->tmem;
  griddep_wait();
  griddep_launch_dependents();

  if (warp == 0) {
    if (lane == 0) {
      // w is read once when one tile of tokens covers them all
      const uint64_t pw = p.stream ? policy_evict_first() : policy_evict_normal();
      const uint64_t px = policy_evict_normal();
      SegIter it(p.s, cta);
      Seg g;
      int st = 0, issued = 0;
      uint32_t ph = 0;
      bool ok = true;
      while (ok && it.next(g)) {
        const int ft = g.t / p.MT, mt = g.t - ft * p.MT, f0 = ft * width, m0 = mt * NT;
        for (int kc = g.k0; kc < g.k1; ++kc) {
          if (!dn_wait(&bars->empty[st], ph ^ 1, abort)) {
            dn_fail(bars, status);
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&bars->full[st], stage_bytes);
          ++issued;
          const uint32_t a = smem_addr(ring + (size_t)st * stage_bytes);
          const int k = kc * kDnChunk;
          if (!p.kn) {
            tma_2d(a, &mw, k, f0, &bars->full[st], pw);
            if (p.gated) tma_2d(a + kDnBytesA / 2, &mw2, k, f0, &bars->full[st], pw);
            else tma_2d(a + kDnBytesA / 2, &mw, k, f0 + kDnHalf, &bars->full[st], pw);
          } else {
            tma_2d(a, &mw, f0, k, &bars->full[st], pw);
            tma_2d(a + 8192, &mw, f0 + 64, k, &bars->full[st], pw);
            const CUtensorMap* m2 = p.gated ? &mw2 : &mw;
            const int f1 = p.gated ? f0 : f0 + kDnHalf;
            tma_2d(a + 16384, m2, f1, k, &bars->full[st], pw);
            tma_2d(a + 24576, m2, f1 + 64, k, &bars->full[st], pw);
          }
          tma_2d(a + kDnBytesA, &mx, k, m0, &bars->full[st], px);
          if (++st == S) {
            st = 0;
            ph ^= 1;
          }
        }
      }
      // no copy of this CTA is in flight when it ends: the last S stages have come
      const int n = issued < S ? issued : S;
      for (int i = 0; i < n; ++i) {
        if (--st < 0) {
          st = S - 1;
          ph ^= 1;
        }
        for (uint32_t w = 0; w < kWaitTries && !mbar_try_wait(&bars->full[st], ph); ++w) {}
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t desc = mma_desc(NT, p.bf16, p.kn);
      SegIter it(p.s, cta);
      Seg g;
      int st = 0, buf = 0;
      uint32_t ph = 0, tph = 0;
      bool ok = true, open = false;
      while (ok && it.next(g)) {
        if (!dn_wait(&bars->tempty[buf], tph ^ 1, abort)) {
          dn_fail(bars, status);
          break;
        }
        tc_after_sync();
        const uint32_t d0 = tmem + buf * 2 * NT, d1 = d0 + NT;
        for (int kc = g.k0; kc < g.k1; ++kc) {
          if (!dn_wait(&bars->full[st], ph, abort)) {
            dn_fail(bars, status);
            ok = false;
            break;
          }
          tc_after_sync();
          const uint32_t a = smem_addr(ring + (size_t)st * stage_bytes);
          dn_stage_products(a, a + kDnBytesA, d0, d1, desc, p.kn, kc == g.k0);
          mma_commit(&bars->empty[st]);
          open = true;
          if (++st == S) {
            st = 0;
            ph ^= 1;
          }
        }
        if (!ok) break;
        mma_commit(&bars->tfull[buf]);
        if (++buf == p.acc_bufs) {
          buf = 0;
          tph ^= 1;
        }
      }
      if (open) {  // every product is done before TMEM is given back
        mma_commit(&bars->drain);
        for (uint32_t w = 0; w < kWaitTries && !mbar_try_wait(&bars->drain, 0); ++w) {}
      }
    }
  } else if (warp >= 4) {
    // lanes 32 (warp % 4) ... are this warp's; of the two warps that have them, with w_mul each takes
    // every other 16 tokens, without it one takes each 128 features
    const int q = warp & 3, half = (warp - 4) >> 2, r = q * 32 + lane, etid = tid - 128;
    const int step = p.gated ? 32 : 16, begin = p.gated ? 16 * half : 0;
    SegIter it(p.s, cta);
    Seg g;
    int buf = 0;
    uint32_t tph = 0;
    while (it.next(g)) {
      const bool ok = dn_wait(&bars->tfull[buf], tph, abort);
      if (!ok) dn_fail(bars, status);
      if (dn_any(1, kDnEpi, !ok)) break;  // one decision for the warps: they meet at barriers below
      tc_after_sync();
      const int ft = g.t / p.MT, mt = g.t - ft * p.MT, m0 = mt * NT;
      const int nt = p.M - m0 < NT ? p.M - m0 : NT;  // tokens of this tile
      const int feat = ft * width + (p.gated ? 0 : half * kDnHalf) + r;
      const bool on = feat < p.N;
      const uint32_t d0 = tmem + ((uint32_t)(q * 32) << 16) + buf * 2 * NT + (p.gated ? 0 : half * NT);
      const int parts = p.s.parts(g.t);
      const float ba = p.bias && on ? ld16(p.bias, feat, p.bf16) : 0.f;
      const float bb = p.bias_mul && on ? ld16(p.bias_mul, feat, p.bf16) : 0.f;
      const size_t seg_floats = (size_t)2 * NT * 128;
      float* mine = p.part + ((size_t)(g.t - p.s.dp) + cta) * seg_floats + r;  // used where parts > 1
      if (!p.gated) mine += half * NT * 128;
      for (int n0 = begin; n0 < nt; n0 += step) {
        float v[16], m[16];
        tmem_ld(d0 + n0, v);
        if (p.gated) tmem_ld(d0 + NT + n0, m);
        tmem_wait(v);
        if (p.gated) tmem_wait(m);
        if (parts == 1) {
          if (on) linear_store(p, feat, m0 + n0, nt - n0, ba, bb, v, m, p.gated);
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if (n0 + i < nt) {
              __stcg(mine + (n0 + i) * 128, v[i]);
              if (p.gated) __stcg(mine + (NT + n0 + i) * 128, m[i]);
            }
          }
        }
        __syncwarp();
      }
      tc_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->tempty[buf]);
      if (parts > 1 && dn_last_share(&p.head->cnt[g.t - p.s.dp], parts, bars, etid) && on) {
        const float* from = p.part + ((size_t)(g.t - p.s.dp) + p.s.first(g.t)) * seg_floats + r;
        if (!p.gated) from += half * NT * 128;
        for (int n0 = begin; n0 < nt; n0 += step) {
          float v[16], m[16];
          sum_shares(from + n0 * 128, seg_floats, parts, nt - n0, v);
          if (p.gated) sum_shares(from + (NT + n0) * 128, seg_floats, parts, nt - n0, m);
          linear_store(p, feat, m0 + n0, nt - n0, ba, bb, v, m, p.gated);
        }
      }
      if (++buf == p.acc_bufs) {
        buf = 0;
        tph ^= 1;
      }
    }
  }
  __syncwarp();
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  if (warp == 2) tmem_free(tmem, p.tmem_cols);
}

struct LinearPlan {
  int NT, MT, FT;
  Sched s;
};

LinearPlan linear_plan(int M, int N, int K, bool gated, int sms) {
  LinearPlan l;
  // equal tiles of at most 256 tokens, a multiple of 16
  l.MT = (M + 255) / 256;
  l.NT = ((M + l.MT - 1) / l.MT + 15) / 16 * 16;
  l.MT = (M + l.NT - 1) / l.NT;
  const int width = gated ? kDnHalf : 2 * kDnHalf;
  l.FT = (N + width - 1) / width;
  l.s = Sched::make(l.FT * l.MT, (K + kDnChunk - 1) / kDnChunk, sms);
  return l;
}

constexpr size_t kHeadBytes = (sizeof(DenseHead) + 255) / 256 * 256;

}  // namespace

size_t linear_ws_bytes(int M, int N, int K, bool gated, int sms) {
  if (M == 0) return kHeadBytes;
  const LinearPlan l = linear_plan(M, N, K, gated, sms);
  return kHeadBytes + (size_t)l.s.segments() * 2 * l.NT * 128 * sizeof(float);
}

cudaError_t launch_linear(const LinearCall& c, void* ws, int sms, int smem_optin, cudaStream_t st) {
  const bool gated = c.w_mul != nullptr;
  const LinearPlan l = linear_plan(c.M, c.N, c.K, gated, sms);
  CUtensorMap mw, mw2, mx;
  const uint64_t cols = c.kn ? c.N : c.K, rows = c.kn ? c.K : c.N;
  const uint32_t box = c.kn ? kDnChunk : kDnHalf;
  cudaError_t e = dense_map(&mw, c.w, c.bf16, cols, rows, c.w_stride, 0, 0, box);
  if (e != cudaSuccess) return e;
  mw2 = mw;
  if (gated) e = dense_map(&mw2, c.w_mul, c.bf16, cols, rows, c.w_mul_stride, 0, 0, box);
  if (e == cudaSuccess) e = dense_map(&mx, c.x, c.bf16, c.K, c.M, c.K, 0, 0, l.NT);
  if (e != cudaSuccess) return e;
  LinearArgs p;
  p.M = c.M;
  p.N = c.N;
  p.MT = l.MT;
  p.NT = l.NT;
  p.gated = gated;
  p.bf16 = c.bf16;
  p.kn = c.kn;
  p.act = c.act;
  p.out_f32 = c.out_f32;
  p.s = l.s;
  p.bias = c.bias;
  p.bias_mul = c.bias_mul;
  p.residual = c.residual;
  p.y = c.y;
  p.head = reinterpret_cast<DenseHead*>(ws);
  p.part = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(ws) + kHeadBytes);
  const int stage = kDnBytesA + l.NT * 128;
  int S = (smem_optin - 1024 - (int)sizeof(DenseBars)) / stage;
  p.stages = S > kDnMaxStages ? kDnMaxStages : S;
  p.acc_bufs = l.NT <= 128 ? 2 : 1;
  p.tmem_cols = 32;
  while (p.tmem_cols < 2 * l.NT * p.acc_bufs) p.tmem_cols *= 2;
  p.stream = l.MT == 1;
  const size_t smem = 1024 + (size_t)p.stages * stage + sizeof(DenseBars);
  e = cudaFuncSetAttribute(linear_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(l.s.ctas());
  cfg.blockDim = dim3(kDnThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, linear_kernel, mw, mw2, mx, p);
}

}  // namespace sesg
