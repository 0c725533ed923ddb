// A whole mixture-of-experts layer with uncompressed 16-bit SwiGLU experts on up to 64 tokens,
// in one kernel:
//
//   l = x Wr, top-k softmax                                     (route)
//   h = SiLU(x G^T) * (x U^T) for every (token, expert) pair       (first phase)
//   y = sum of weight * (h D) over a token's experts               (second phase, join)
//
// With so few tokens the layer is bound by HBM: every active expert's 3 f d weights are read
// once and stream through tcgen05 as the 128-row operand (dense.cuh); an expert's own tokens
// are gathered as the other one.  One CTA per SM stays for the whole layer; three barriers over
// the grid order its phases (cooperative launch, bounded waits), and at the second one the TMA
// warp already streams the next phase's weights.
//
// h goes to the second phase as two 16-bit values, hi + lo, in two columns of the same
// product: h = hi + lo to 2^-16 (bf16) or 2^-22 (fp16), so that y loses nothing to the operand's
// type, at no cost in bytes from HBM (fp16: |h| > 65504 is infinite, as in fp16 arithmetic).
// Every sum has a fixed order.
#include "dense.cuh"
#include "dense_params.cuh"
#include "layer_plan.h"

namespace sesg {

namespace {

constexpr int kMaxExperts = 256;
constexpr int kMaxActive = kMaxExperts + 8;
constexpr int kMaxPairSlots = 16;                // k + shared experts of a token, at most
constexpr int kJoinGroups = kDnThreads / kDnHalf;

struct LayerArgs {
  int B, d, f, E, k, ns, renorm, rmsnorm, bf16;
  const void *x, *w_router, *residual;
  void* y;
  int32_t* user_idx;
  float* user_w;
  DenseHead* head;
  float* logits;       // [B][slices][E]
  int* top_idx;        // [B][k]
  float* top_w;
  unsigned short* h;   // [groups][hi, lo][8][f]
  float* part;         // first phase: [segment][gate, up][64][128]; second: [segment][B][256]
  float* ysum;         // [sum row][d]
  size_t cut;          // floats from ysum to part
  float* yrow;         // [B][d] sums before RMSNorm
  float* ysq;          // [B][128 features][4 warps] their squares
  int slots;           // 8 * max_groups
  int rows;            // features of a tile of the first phase
  int early;           // tiles of the first phase that stay whole and start before the routing
  int slices;          // router: CTAs per token
  int block_rows, block_vecs, blocks;  // log2 of the rows of a block, its vectors, blocks that a CTA's threads take at a time
  int sum_step;        // threads of the first step of the sums, a multiple of E
  int stages, stage_bytes, a_bytes;  // a_bytes: of a stage, before the tokens
  uint32_t tries;      // rounds of a wait
  int missing;         // diagnostics: the barrier over the grid that misses an arrival, or -1
};

struct LayerMisc {
  DenseBars bars;
  unsigned long long mask[kMaxExperts];  // tokens of each routed expert
  uint32_t on[kMaxExperts / 32];         // experts with tokens (few tokens)
  short where[kMaxExperts];              // its place among the active ones
  short act[kMaxActive];                 // active experts: shared ones (E + s) first
  short cnt[kMaxActive];                 // ... tokens
  short grp[kMaxActive];                 // ... first group of 8 slots
  short sum[kMaxActive];                 // ... first row of sums
  int n_act;
  int last;
  int fail;
  int idx[kDenseMaxTok * 8];
  float w[kDenseMaxTok * 8];
  short row[kDenseMaxTok * kMaxPairSlots];    // sum row of each (token, choice)
  short place[kDenseMaxTok * kMaxPairSlots];  // active expert of each (token, choice)
  // a token's partial sums: where they begin and their weights
  size_t from[kJoinGroups][kMaxPairSlots * (kDnMaxSplit + 1)];
  float weight[kJoinGroups][kMaxPairSlots * (kDnMaxSplit + 1)];
  int n_from[kJoinGroups];
};

// Arrive at / wait for n CTAs at a barrier over the grid.  All CTAs are resident (cooperative launch).
__device__ __forceinline__ void grid_arrive(unsigned* bar) {
  asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(bar) : "memory");
}
__device__ __forceinline__ bool grid_wait(unsigned* bar, unsigned n, const DenseBars* b) {
  for (uint32_t i = 0; i < b->tries * 1024; ++i) {
    unsigned v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(bar) : "memory");
    if (v >= n) return true;
    if (dn_aborted(b)) return false;
  }
  return false;
}

// Logits of token b over the rows [r0, r1) of the router weight (multiples of 8), to out[E].  A block is one row, or eight
// where E is no multiple of 8: a whole number of vectors of 8 values.  A thread owns one vector of every nrs-th block,
// whose values belong to the same experts each time and, from 8 experts on, to at most two rows.  (Fewer experts: one value
// of every nrs-th row.)  red: 9 kDnThreads
// floats.  Short code on purpose, here and in choose: the kernel fetches it anew in every call (one token of 8 x 1024: 8
// rows in flight, code for odd E of its own and choices in registers 22.4 us, this 20.9; odd E value by value: 61 tokens of
// 19 x 280 54.5 us, this 49.5).
__device__ __forceinline__ void slice_logits(const LayerArgs& p, int b, int r0, int r1, float* out, float* red) {
  constexpr int RU = 4;  // vectors in flight
  const int tid = threadIdx.x, E = p.E, V = p.block_vecs, nrs = p.blocks, rs = tid / V, v = tid - rs * V;
  const unsigned short* x = reinterpret_cast<const unsigned short*>(p.x) + (size_t)b * p.d;
  if (rs < nrs && E < 8) {
    float acc = 0.f;
#pragma unroll 4
    for (int r = r0 + rs; r < r1; r += nrs)
      acc = fmaf(ld16(x, r, p.bf16), ld16(p.w_router, (size_t)r * E + v, p.bf16), acc);
    red[tid] = acc;
  } else if (rs < nrs) {
    float acc[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[i] = 0.f;
    const int ra = v * 8 / E, first = (ra + 1) * E - v * 8;  // values of the vector's first row
    const uint4* w = reinterpret_cast<const uint4*>(p.w_router) + v;
    const int end = r1 >> p.block_rows;
    for (int q = (r0 >> p.block_rows) + rs; q < end; q += nrs * RU) {
      float xa[RU], xc[RU];
      uint4 wv[RU];
#pragma unroll
      for (int u = 0; u < RU; ++u) {
        const int at = q + u * nrs;
        xa[u] = xc[u] = 0.f;
        wv[u] = make_uint4(0, 0, 0, 0);
        if (at < end) {
          const int row = (at << p.block_rows) + ra;
          wv[u] = w[(size_t)at * V];
          xa[u] = ld16(x, row, p.bf16);
          if (p.block_rows) xc[u] = ld16(x, row + (first < 8), p.bf16);
        }
      }
      auto rows = [&](auto value) {
#pragma unroll
        for (int u = 0; u < RU; ++u) {
          const uint32_t w4[4] = {wv[u].x, wv[u].y, wv[u].z, wv[u].w};
#pragma unroll
          for (int i = 0; i < 8; ++i) acc[i] = fmaf(i < first ? xa[u] : xc[u], value(w4[i / 2], i & 1), acc[i]);
        }
      };
      if (p.bf16) rows([](uint32_t w, int hi) { return __uint_as_float(hi ? w & 0xffff0000u : w << 16); });
      else rows([](uint32_t w, int hi) { return from16((unsigned short)(hi ? w >> 16 : w), 0); });
    }
    reinterpret_cast<float4*>(red)[tid * 2] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    reinterpret_cast<float4*>(red)[tid * 2 + 1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
  }
  // [rs][row of a block][expert], summed in two steps
  __syncthreads();
  float* sums = red + 8 * kDnThreads;
  const int step = p.sum_step;
  if (tid < step) {
    float t = 0.f;
#pragma unroll 4
    for (int i = tid; i < (nrs * E) << p.block_rows; i += step) t += red[i];
    sums[tid] = t;
  }
  __syncthreads();
  if (tid < E) {
    float t = 0.f;
#pragma unroll 4
    for (int i = tid; i < step; i += E) t += sums[i];
    __stcg(out + tid, t);
  }
}

// Token b's bit in expert e's mask, in the 32-bit half that has it.
__device__ __forceinline__ void mark_token(LayerMisc& m, int e, int b) {
  atomicOr(reinterpret_cast<uint32_t*>(&m.mask[e]) + (b >> 5), 1u << (b & 31));
}

// One warp: token b's logits (its slices [slices][E] added in order), its k experts by logit descending
// (ties: the lower index; NaN ranks as -inf) and their weights.  A logit's key orders as the logit
// does; an expert that is taken has key 0, below every logit's.  The keys take the first slice's place.  m: where to
// mark the choice, or null.
__device__ __forceinline__ uint32_t logit_key(float l) {
  const uint32_t u = __float_as_uint(l);
  return u >> 31 ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_logit(uint32_t key) {
  return __uint_as_float(key >> 31 ? key & 0x7fffffffu : ~key);
}
__device__ __forceinline__ void choose(const LayerArgs& p, int b, float* slices, int* idx, float* w, LayerMisc* m) {
  const int lane = threadIdx.x & 31;
  uint32_t* keys = reinterpret_cast<uint32_t*>(slices);  // expert e's is lane e % 32's
#pragma unroll 1
  for (int e = lane; e < p.E; e += 32) {
    float s = 0.f;
#pragma unroll 4
    for (int q = 0; q < p.slices; ++q) s += slices[q * p.E + e];
    s += 0.f;  // -0 and +0 are one logit
    keys[e] = logit_key(isnan(s) ? -INFINITY : s);
  }
  float mine = 0.f, top = -INFINITY;  // lane j keeps the j-th choice
  int mine_e = 0;
#pragma unroll 1
  for (int j = 0; j < p.k; ++j) {
    uint32_t best = 0u;
    int at = 0x7fffffff;
#pragma unroll 1
    for (int e = lane; e < p.E; e += 32) {
      const uint32_t key = keys[e];
      if (key > best) {
        best = key;
        at = e;
      }
    }
    const uint32_t most = __reduce_max_sync(0xffffffffu, best);
    const int e = __reduce_min_sync(0xffffffffu, best == most ? at : 0x7fffffff);
    if (lane == (e & 31)) keys[e] = 0u;
    const float v = key_logit(most);
    if (j == 0) top = v;
    if (lane == j) {
      mine = v;
      mine_e = e;
    }
  }
  const float num = expf(mine - top);
  float sum = lane < p.k ? num : 0.f;
  if (!p.renorm) {
#pragma unroll 1
    for (int e = lane; e < p.E; e += 32)
      if (keys[e]) sum += expf(key_logit(keys[e]) - top);
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
  if (lane < p.k) {
    idx[b * p.k + lane] = mine_e;
    w[b * p.k + lane] = num / sum;
    if (m) {
      mark_token(*m, mine_e, b);
      atomicOr(&m->on[mine_e >> 5], 1u << (mine_e & 31));
    }
  }
}

// Whole CTA: n values of other CTAs to shared memory, four of a thread's in flight.
__device__ void gather_logits(const float* from, int n, float* to) {
  for (int i = threadIdx.x; i < n; i += 4 * kDnThreads) {
    float t[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) t[j] = i + j * kDnThreads < n ? __ldcg(from + i + j * kDnThreads) : 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i + j * kDnThreads < n) to[i + j * kDnThreads] = t[j];
  }
}

// Routing of every token into m.idx / m.w.  False: a wait ran out.
__device__ bool route(const LayerArgs& p, LayerMisc& m, float* scratch) {
  const int tid = threadIdx.x, warp = tid >> 5, cta = blockIdx.x;
  const bool few = p.B <= kFewTok;
  if (cta < p.B * p.slices) {
    const int b = cta / p.slices, s = cta - b * p.slices;
    const int len = (p.d / 8 + p.slices - 1) / p.slices * 8;
    const int r0 = s * len, r1 = r0 + len < p.d ? r0 + len : p.d;
    float* out = p.logits + ((size_t)b * p.slices + s) * p.E;
    slice_logits(p, b, r0, r1, out, scratch);
    __syncthreads();
    if (!few) {
      // the token's last slice to come chooses its experts
      if (tid == 0) {
        unsigned old;
        asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(&p.head->tok[b]) : "memory");
        m.last = old == (unsigned)(p.slices - 1);
        if (m.last) p.head->tok[b] = 0u;
      }
      __syncthreads();
      if (m.last) {
        gather_logits(p.logits + (size_t)b * p.slices * p.E, p.slices * p.E, scratch);
        __syncthreads();
        if (warp == 0) {
          choose(p, b, scratch, p.top_idx, p.top_w, nullptr);
        }
      }
      __syncthreads();
    }
  }
  if (tid == 0) {
    if (cta < p.B * p.slices) grid_arrive(&p.head->bar[0]);
    m.fail = !grid_wait(&p.head->bar[0], p.B * p.slices + (p.missing == 0), &m.bars);
  }
  __syncthreads();
  if (m.fail) return false;
  if (few) {
    gather_logits(p.logits, p.B * p.slices * p.E, scratch);
    __syncthreads();
    if (warp < p.B) choose(p, warp, scratch + warp * p.slices * p.E, m.idx, m.w, &m);
  } else {
    for (int i = tid; i < p.B * p.k; i += kDnThreads) {
      m.idx[i] = __ldcg(p.top_idx + i);
      m.w[i] = __ldcg(p.top_w + i);
    }
  }
  __syncthreads();
  if (cta == 0) {
    for (int i = tid; i < p.B * p.k; i += kDnThreads) {
      if (p.user_idx) p.user_idx[i] = m.idx[i];
      if (p.user_w) p.user_w[i] = m.w[i];
    }
  }
  return true;
}

// The active experts, their tokens in ascending order, and the slot of every (token, choice).
__device__ void make_lists(const LayerArgs& p, LayerMisc& m, uint8_t* tok) {
  const int tid = threadIdx.x, lane = tid & 31;
  const int pairs = p.B * p.k, gs = (p.B + 7) / 8;
  if (p.B <= kFewTok) {
    // One group of 8 slots for each active expert, in the order of the experts; the routing has marked the
    // masks.  One thread for each (token, choice).
    if (tid < pairs + p.B * p.ns) {
      int b, j, a, before;
      if (tid < pairs) {
        b = tid / p.k;
        j = tid - b * p.k;
        const int e = m.idx[tid];
        a = p.ns + __popc(m.on[e >> 5] & ((1u << (e & 31)) - 1));
        for (int i = 0; i < e >> 5; ++i) a += __popc(m.on[i]);
        const unsigned long long mask = m.mask[e];
        before = __popcll(mask & ((1ull << b) - 1));
        if (before == 0) {
          m.act[a] = (short)e;
          m.cnt[a] = (short)__popcll(mask);
          m.grp[a] = (short)a;
          m.sum[a] = (short)(8 * a);
        }
      } else {
        a = (tid - pairs) / p.B;
        b = before = (tid - pairs) - a * p.B;
        j = p.k + a;
        if (b == 0) {
          m.act[a] = (short)(p.E + a);
          m.cnt[a] = (short)p.B;
          m.grp[a] = (short)a;
          m.sum[a] = (short)(8 * a);
        }
      }
      tok[a * 8 + before] = (uint8_t)b;
      m.row[b * kMaxPairSlots + j] = (short)(a * 8 + before);
      m.place[b * kMaxPairSlots + j] = (short)a;
    }
    if (tid == kDnThreads - 1) {
      int n = p.ns;
      for (int i = 0; i < (p.E + 31) / 32; ++i) n += __popc(m.on[i]);
      m.n_act = n;
    }
    __syncthreads();
    return;
  }
  for (int i = tid; i < pairs; i += kDnThreads) mark_token(m, m.idx[i], i / p.k);
  __syncthreads();
  if (tid < 32) {
    if (lane < p.ns) {
      m.act[lane] = (short)(p.E + lane);
      m.cnt[lane] = (short)p.B;
      m.grp[lane] = (short)(lane * gs);
      m.sum[lane] = (short)(lane * p.B);
    }
    int na = p.ns, ng = p.ns * gs, nt = p.ns * p.B;
    for (int base = 0; base < p.E; base += 32) {
      const int e = base + lane;
      const int n = e < p.E ? __popcll(m.mask[e]) : 0, g = (n + 7) / 8;
      const uint32_t on = __ballot_sync(0xffffffffu, n > 0);
      int sg = g << 16 | n;  // at most 64 groups and 32 * 64 tokens in a step
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, sg, off);
        if (lane >= off) sg += o;
      }
      if (n > 0) {
        const int a = na + __popc(on & ((1u << lane) - 1));
        m.act[a] = (short)e;
        m.cnt[a] = (short)n;
        m.grp[a] = (short)(ng + (sg >> 16) - g);
        m.sum[a] = (short)(nt + (sg & 0xffff) - n);
        m.where[e] = (short)a;
      }
      na += __popc(on);
      sg = __shfl_sync(0xffffffffu, sg, 31);
      ng += sg >> 16;
      nt += sg & 0xffff;
    }
    if (lane == 0) m.n_act = na;
  }
  __syncthreads();
  for (int i = tid; i < pairs; i += kDnThreads) {
    const int b = i / p.k, j = i - b * p.k, e = m.idx[i], a = m.where[e];
    const int before = __popcll(m.mask[e] & ((1ull << b) - 1));
    tok[m.grp[a] * 8 + before] = (uint8_t)b;
    m.row[b * kMaxPairSlots + j] = (short)(m.sum[a] + before);
    m.place[b * kMaxPairSlots + j] = (short)a;
  }
  for (int i = tid; i < p.B * p.ns; i += kDnThreads) {
    const int s = i / p.B, b = i - s * p.B;
    tok[s * gs * 8 + b] = (uint8_t)b;
    m.row[b * kMaxPairSlots + p.k + s] = (short)(s * p.B + b);
    m.place[b * kMaxPairSlots + p.k + s] = (short)s;
  }
  __syncthreads();
}

// h of W tokens of one feature (n of them exist), from their sums of gate and up, to slots slot ...
template <int W>
__device__ __forceinline__ void store_h(const LayerArgs& p, int slot, int n, int feat, const float (&g)[W],
                                        const float (&u)[W]) {
  unsigned short hi[W], lo[W];
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const float h = silu_f(g[i]) * u[i];
    hi[i] = to16(h, p.bf16);
    const float hf = from16(hi[i], p.bf16);
    lo[i] = isfinite(hf) ? to16(h - hf, p.bf16) : (unsigned short)0;
  }
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const int s = slot + i;
    unsigned short* to = p.h + ((size_t)(s >> 3) * 16 + (s & 7)) * p.f + feat;
    if (i < n) {
      to[0] = hi[i];
      to[(size_t)8 * p.f] = lo[i];
    }
  }
}

// First phase's epilogue of W tokens (n of them exist) of a tile that one CTA did whole, ...
template <int W>
__device__ __forceinline__ void whole_h(const LayerArgs& p, uint32_t t, int slot, int n, int feat) {
  float g[W], u[W];
  tmem_ld(t, g);
  tmem_ld(t + 128, u);
  tmem_wait(g);
  tmem_wait(u);
  if (feat < p.f) store_h(p, slot, n, feat, g, u);
  __syncwarp();
}
// ... of a share of a split tile, to its place among the partial sums, ...
template <int W>
__device__ __forceinline__ void share_h(uint32_t t, int n, float* to) {
  float g[W], u[W];
  tmem_ld(t, g);
  tmem_ld(t + 128, u);
  tmem_wait(g);
  tmem_wait(u);
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if (i < n) {
      __stcg(to + i * kDnHalf, g[i]);
      __stcg(to + (kDenseMaxTok + i) * kDnHalf, u[i]);
    }
  }
  __syncwarp();
}
// ... and of the shares together.
template <int W>
__device__ __forceinline__ void joined_h(const LayerArgs& p, const float* from, int parts, int slot, int n, int feat) {
  float g[W], u[W];
  sum_shares(from, kDenseMaxTok * kDnHalf, kPartFloats, parts, n, g, u);
  store_h(p, slot, n, feat, g, u);
}

struct LayerMaps {
  CUtensorMap gate, up, down;        // routed experts
  CUtensorMap sgate, sup, sdown;     // shared experts
  CUtensorMap x, h;
};

// WIDE: chunks of 64 k in a stage of the first phase.
template <int WIDE>
__global__ void __launch_bounds__(kDnThreads, 1)
dense_layer_kernel(const __grid_constant__ LayerMaps maps, const LayerArgs p) {
  extern __shared__ uint8_t raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  LayerMisc& m = *reinterpret_cast<LayerMisc*>(ring + (size_t)p.stages * p.stage_bytes);
  uint8_t* tok = reinterpret_cast<uint8_t*>(&m + 1);
  DenseBars* bars = &m.bars;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, cta = blockIdx.x;
  const int S = p.stages;
  const int FT = (p.f + p.rows - 1) / p.rows, DT = (p.d + 2 * kDnHalf - 1) / (2 * kDnHalf);
  const int chunks = (p.d + kDnChunk - 1) / kDnChunk;
  const int KC1 = (chunks + WIDE - 1) / WIDE, KC2 = (p.f + kDnChunk - 1) / kDnChunk;  // stages of a tile
  const uint32_t ring_at = smem_addr(ring);
  const uint32_t half_a = p.rows * 128;  // bytes of a chunk of gate rows, or of up rows
  const uint32_t x_bytes = (p.B + 7) / 8 * 1024;  // ... of the tokens'
  const uint32_t a_bytes = WIDE == 1 ? kDnBytesA : p.a_bytes;
  int* status = &p.head->ctrl.status;

  if (tid == 0) {
    dn_init_bars(bars, p.tries);
    m.fail = 0;
  }
  if (warp == 2) tmem_alloc(&bars->tmem, 512);
  if (warp == 3 && lane < 8) tma_prefetch_map(&maps.gate + lane);
  // make_lists starts from no tokens
  for (int e = tid; e < p.E; e += kDnThreads) m.mask[e] = 0ull;
  if (tid < kMaxExperts / 32) m.on[tid] = 0u;
  for (int i = tid; i < p.slots; i += kDnThreads) tok[i] = (uint8_t)p.B;
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  const uint32_t tmem = bars->tmem;
  griddep_launch_dependents();  // the next call's CTAs take the SMs that this kernel's leave

  // Chunk kc of a tile of the first phase, into a stage.  The shared experts' tiles come first: they do not depend on the
  // routing.
  const uint64_t pw = policy_evict_first(), px = policy_evict_normal();
  auto load_gate_up = [&](int t, int kc, int stage) {
    const int a = t / FT, f0 = (t - a * FT) * p.rows;
    const int c0 = kc * WIDE, c1 = WIDE == 1 ? c0 + 1 : c0 + WIDE < chunks ? c0 + WIDE : chunks;
    const bool routed = a >= p.ns;
    const int z = routed ? m.act[a] : a, n4 = ((routed ? m.cnt[a] : p.B) + 3) / 4;
    uint64_t* full = &bars->full[stage];
    mbar_arrive_expect_tx(full, (c1 - c0) * (2 * half_a + n4 * 512));
    uint32_t at = ring_at + stage * p.stage_bytes, xat = at + a_bytes;
#pragma unroll 1
    for (int c = c0; c < c1; ++c, at += 2 * half_a, xat += x_bytes) {
      const int k = c * kDnChunk;
      tma_3d(at, routed ? &maps.gate : &maps.sgate, k, f0, z, full, pw);
      tma_3d(at + half_a, routed ? &maps.up : &maps.sup, k, f0, z, full, pw);
      if (routed) {
        const uint8_t* q = tok + m.grp[a] * 8;
        for (int r = 0; r < n4; ++r, q += 4) tma_rows4(xat + r * 512, &maps.x, k, q[0], q[1], q[2], q[3], full, px);
      } else {
        for (int r = 0; r < n4; ++r)
          tma_rows4(xat + r * 512, &maps.x, k, 4 * r, 4 * r + 1, 4 * r + 2, 4 * r + 3, full, px);
      }
    }
  };
  // The first stages of whole ones are on their way while the tokens are routed, whose scratch is the last stage.
  int sent = 0;
  if (warp == 0 && elect_one()) {
    for (int t = cta; t < p.early; t += gridDim.x)
      for (int kc = 0; kc < KC1 && sent < S - 1; ++kc) load_gate_up(t, kc, sent++);
    // ... and the first of their down rows on the way to L2
    for (int i = cta, n = 0; i < p.ns * DT * KC2 && n < 4; i += gridDim.x, ++n) {
      const int t = i / KC2, z = t / DT;
      for (int j = 0; j < 4; ++j)
        tma_prefetch_3d(&maps.sdown, (t - z * DT) * 2 * kDnHalf + 64 * j, (i - t * KC2) * kDnChunk, z);
    }
  }
  __syncwarp();

  const bool ok = route(p, m, reinterpret_cast<float*>(ring + (size_t)(S - 1) * p.stage_bytes));
  if (!ok && tid == 0) dn_fail(bars, status);
  if (ok) make_lists(p, m, tok);
  // the ring was scratch of the router: its generic accesses come before the copies into it
  fence_proxy_async_smem();
  __syncthreads();

  const Sched s1 = Sched::make(m.n_act * FT, KC1, gridDim.x, p.early);
  const Sched s2 = Sched::make(m.n_act * DT, KC2, gridDim.x, 0);

  // join: every token's experts and their shares, in order.  A unit is 128 features of a token; each four
  // warps take one at a time, the first of them lists where the token's sums lie.
  const int grp = tid / kDnHalf, gtid = tid - grp * kDnHalf, HT = (p.d + kDnHalf - 1) / kDnHalf;
  const int u0 = cta * kJoinGroups + grp, ustep = gridDim.x * kJoinGroups;
  auto list_sums = [&](int u, int grp) {
    const int b = u / HT, dt = (u - b * HT) / 2;
    int parts = 0;
    size_t from = 0, step = 0;
    if (lane < p.k + p.ns) {
      const int a = m.place[b * kMaxPairSlots + lane], row = m.row[b * kMaxPairSlots + lane], t = a * DT + dt;
      parts = s2.parts(t);
      from = (size_t)row * p.d;
      if (parts > 1) {
        step = (size_t)p.B * 2 * kDnHalf;
        from = p.cut + (t - s2.dp + s2.first(t)) * step + (row - m.sum[a]) * 2 * kDnHalf - dt * 2 * kDnHalf;
      }
    }
    int end = parts;
#pragma unroll
    for (int off = 1; off < 16; off <<= 1) {
      const int o = __shfl_up_sync(0xffffffffu, end, off);
      if (lane >= off) end += o;
    }
    for (int s = 0; s < parts; ++s) {
      m.from[grp][end - parts + s] = from + s * step;
      m.weight[grp][end - parts + s] = lane < p.k ? m.w[b * p.k + lane] : 1.f;
    }
    if (lane == 15) m.n_from[grp] = end;
    __syncwarp();
  };
  if (!ok) {
    // no copy is in flight when the CTA ends
    for (int i = 0; i < sent; ++i)
      dn_drain(&bars->full[i], 0, kWaitTries);
  } else if (warp == 0) {
    if (elect_one()) {
      int st = 0, issued = sent;
      uint32_t ph = 0;
      auto advance = [&](int& s, uint32_t& h) {
        if (++s == S) {
          s = 0;
          h ^= 1;
        }
      };
      Seg g;
      bool go = true;
      int skip = sent;  // chunks that are on their way
      SegIter it(s1, cta);
      while (go && it.next(g)) {
        for (int kc = g.k0; kc < g.k1; ++kc) {
          if (skip > 0) {
            --skip;
            advance(st, ph);
            continue;
          }
          if (!dn_wait(&bars->empty[st], ph ^ 1, bars)) {
            dn_fail(bars, status);
            go = false;
            break;
          }
          load_gate_up(g.t, kc, st);
          ++issued;
          advance(st, ph);
        }
      }
      // second phase: the weights of the first stages are asked for before the grid's h is there
      auto load_down = [&](const Seg& q, int kc, int stage) {
        const int a = q.t / DT, d0 = (q.t - a * DT) * 2 * kDnHalf, e = m.act[a], ng = (m.cnt[a] + 7) / 8;
        const bool sh = e >= p.E;
        const CUtensorMap* md = sh ? &maps.sdown : &maps.down;
        uint64_t* full = &bars->full[stage];
        mbar_arrive_expect_tx(full, kDnBytesA + ng * 2048);
        const uint32_t at = ring_at + stage * p.stage_bytes;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          tma_3d(at + i * 8192, md, d0 + 64 * i, kc * kDnChunk, sh ? e - p.E : e, full, pw);
      };
      auto load_h = [&](const Seg& q, int kc, int stage) {
        const int a = q.t / DT, ng = (m.cnt[a] + 7) / 8, row = m.grp[a] * 16;
        const uint32_t at = ring_at + stage * p.stage_bytes + a_bytes;
        for (int i = 0; i < ng; ++i)
          tma_2d(at + i * 2048, &maps.h, kc * kDnChunk, row + 16 * i, &bars->full[stage], px);
      };
      SegIter w2(s2, cta), h2(s2, cta);
      Seg gw, gh;
      bool more = go && w2.next(gw);
      int kw = more ? gw.k0 : 0, hs = st, ahead = 0;
      uint32_t hp = ph;
      bool hmore = more && h2.next(gh), waited = false;
      int kh = hmore ? gh.k0 : 0;
      while (go && hmore) {
        // weights as far ahead as there are stages, then the h of the oldest of them
        while (more && ahead < (waited ? 1 : S)) {
          if (!dn_wait(&bars->empty[st], ph ^ 1, bars)) {
            dn_fail(bars, status);
            go = false;
            break;
          }
          load_down(gw, kw, st);
          ++issued;
          ++ahead;
          advance(st, ph);
          if (++kw == gw.k1) {
            more = w2.next(gw);
            if (more) kw = gw.k0;
          }
        }
        if (!go) break;
        if (!waited) {
          waited = true;
          if (!grid_wait(&p.head->bar[1], gridDim.x + (p.missing == 1), bars)) {
            dn_fail(bars, status);
            break;
          }
          fence_proxy_async_all();  // h was stored by threads, and is read by the async proxy
        }
        load_h(gh, kh, hs);
        --ahead;
        advance(hs, hp);
        if (++kh == gh.k1) {
          hmore = h2.next(gh);
          if (hmore) kh = gh.k0;
        }
      }
      // no copy of this CTA is in flight when it ends.  Stages whose h was never asked for (an
      // abort) cannot complete: their weights have come long before this bounded wait is over.
      const int n = issued < S ? issued : S;
      for (int i = 0; i < n; ++i) {
        if (--st < 0) {
          st = S - 1;
          ph ^= 1;
        }
        dn_drain(&bars->full[st], ph, dn_aborted(bars) ? 8 : kWaitTries);
      }
    }
  } else if (warp == 2 || warp == 3) {
    // the join's first units are listed while the other warps work
    for (int i = warp - 2; i < kJoinGroups; i += 2)
      if (cta * kJoinGroups + i < p.B * HT) list_sums(cta * kJoinGroups + i, i);
  } else if (warp == 1) {
    if (elect_one()) {
      int st = 0, buf = 0;
      uint32_t ph = 0, tph = 0;
      bool go = true, open = false;
      Seg g;
#pragma unroll 1
      for (int phase = 0; phase < 2 && go; ++phase) {
        const int TT = phase ? DT : FT;
        const uint32_t second = phase ? kDnBytesA / 2 : half_a;
        SegIter it(phase ? s2 : s1, cta);
        while (go && it.next(g)) {
          const int n = m.cnt[g.t / TT];
          const uint32_t desc = mma_desc(phase ? (n + 7) / 8 * 16 : (n + 15) / 16 * 16, p.bf16, phase);
          if (!dn_wait(&bars->tempty[buf], tph ^ 1, bars)) {
            dn_fail(bars, status);
            go = false;
            break;
          }
          tc_after_sync();
          const uint32_t d0 = tmem + buf * 256;
          for (int kc = g.k0; kc < g.k1; ++kc) {
            if (!dn_wait(&bars->full[st], ph, bars)) {
              dn_fail(bars, status);
              go = false;
              break;
            }
            tc_after_sync();
            uint32_t a = ring_at + st * p.stage_bytes, x = a + a_bytes;
            const int left = chunks - kc * WIDE, nc = WIDE == 1 || phase ? 1 : left < WIDE ? left : WIDE;
#pragma unroll 1
            for (int c = 0; c < nc; ++c, a += 2 * half_a, x += x_bytes)
              dn_stage_products(a, x, d0, d0 + 128, desc, phase != 0, c == 0 && kc == g.k0, true, second);
            mma_commit(&bars->empty[st]);
            open = true;
            if (++st == S) {
              st = 0;
              ph ^= 1;
            }
          }
          if (!go) break;
          mma_commit(&bars->tfull[buf]);
          buf ^= 1;
          tph ^= buf == 0;
        }
      }
      if (open) {
        mma_commit(&bars->drain);
        dn_drain(&bars->drain, 0, kWaitTries);
      }
    }
  } else if (warp >= 4) {
    // lanes 32 (warp % 4) ... are this warp's; of the two warps that have them, in the first phase each takes
    // every other 8 tokens, in the second each takes 128 features
    const int q = warp & 3, half = (warp - 4) >> 2, r = q * 32 + lane, etid = tid - 128;
    int buf = 0;
    uint32_t tph = 0;
    bool go = true;
    Seg g;
    {
      SegIter it(s1, cta);
      while (it.next(g)) {
        const bool good = dn_wait(&bars->tfull[buf], tph, bars);
        if (!good) dn_fail(bars, status);
        if (dn_any(1, kDnEpi, !good)) {
          go = false;
          break;
        }
        tc_after_sync();
        const int a = g.t / FT, n = m.cnt[a], slot = m.grp[a] * 8;
        const int feat = r < p.rows ? (g.t - a * FT) * p.rows + r : p.f;  // p.f: none
        const uint32_t t0 = tmem + ((uint32_t)(q * 32) << 16) + buf * 256;
        const int parts = s1.parts(g.t);
        float* mine = p.part + ((size_t)(g.t - s1.dp) + cta) * kPartFloats + r;  // used where parts > 1
        // up to two tokens in code of their own: a kernel this short pays for every line of code it fetches
        if (n <= 2) {
          if (half == 0) {
            if (parts == 1) whole_h<2>(p, t0, slot, n, feat);
            else share_h<2>(t0, n, mine);
          }
        } else {
          for (int n0 = 8 * half; n0 < n; n0 += 16) {
            if (parts == 1) whole_h<8>(p, t0 + n0, slot + n0, n - n0, feat);
            else share_h<8>(t0 + n0, n - n0, mine + n0 * kDnHalf);
          }
        }
        tc_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->tempty[buf]);
        if (parts > 1 && dn_last_share(&p.head->cnt[g.t - s1.dp], parts, bars, etid) && feat < p.f) {
          const float* from = p.part + ((size_t)(g.t - s1.dp) + s1.first(g.t)) * kPartFloats + r;
          if (n <= 2) {
            if (half == 0) joined_h<2>(p, from, parts, slot, n, feat);
          } else {
            for (int n0 = 8 * half; n0 < n; n0 += 16)
              joined_h<8>(p, from + n0 * kDnHalf, parts, slot + n0, n - n0, feat);
          }
        }
        buf ^= 1;
        tph ^= buf == 0;
      }
    }
    __syncwarp();
    if (go) {
      // this CTA's h: the barrier and the count's release order its stores before what the other CTAs do
      // once they have seen the count
      named_barrier(1, kDnEpi);
      if (etid == 0) grid_arrive(&p.head->bar[1]);
      SegIter it(s2, cta);
      while (it.next(g)) {
        const bool good = dn_wait(&bars->tfull[buf], tph, bars);
        if (!good) dn_fail(bars, status);
        if (dn_any(1, kDnEpi, !good)) break;
        tc_after_sync();
        const int a = g.t / DT, n = m.cnt[a];
        const int feat = (g.t - a * DT) * 2 * kDnHalf + half * kDnHalf + r;
        const uint32_t t0 = tmem + ((uint32_t)(q * 32) << 16) + buf * 256 + half * 128;
        // a whole tile's sums to the tokens' rows, a share's to its place among the shares
        const bool cut = s2.parts(g.t) > 1;
        const size_t step = cut ? 2 * kDnHalf : p.d;
        float* out = cut ? p.part + (size_t)(g.t - s2.dp + cta) * p.B * 2 * kDnHalf + half * kDnHalf + r
                         : p.ysum + (size_t)m.sum[a] * p.d + feat;
        for (int n0 = 0; n0 < n; n0 += 8) {  // columns: 8 tokens' hi, then their lo
          float v[16];
          tmem_ld(t0 + 2 * n0, v);
          tmem_wait(v);
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (n0 + i < n && feat < p.d) __stcg(out + (n0 + i) * step, v[i] + v[i + 8]);
          __syncwarp();
        }
        tc_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->tempty[buf]);
        buf ^= 1;
        tph ^= buf == 0;
      }
    }
  }
  __syncwarp();
  tc_before_sync();
  __syncthreads();
  tc_after_sync();
  if (warp == 2) tmem_free(tmem, 512);

  if (tid == 0) {
    if (!dn_aborted(bars)) {
      grid_arrive(&p.head->bar[2]);
      if (!grid_wait(&p.head->bar[2], gridDim.x + (p.missing == 2), bars)) dn_fail(bars, status);
    }
    m.fail = dn_aborted(bars);
  }
  __syncthreads();
  const bool failed = m.fail;
  const int units = failed ? 0 : p.B * HT;
  for (int u = u0; u < units; u += ustep) {
    const int b = u / HT, feat = (u - b * HT) * kDnHalf + gtid;
    if (u != u0) {
      named_barrier(2 + grp, kDnHalf);
      if (gtid < 32) list_sums(u, grp);
      named_barrier(2 + grp, kDnHalf);
    }
    float acc = 0.f;
    if (feat < p.d) {
      const int n = m.n_from[grp];
      const float r = p.residual ? ld16(p.residual, (size_t)b * p.d + feat, p.bf16) : 0.f;
#pragma unroll 1
      for (int i = 0; i < n; i += 16) {
        float t[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) t[j] = i + j < n ? __ldcg(p.ysum + m.from[grp][i + j] + feat) : 0.f;
#pragma unroll
        for (int j = 0; j < 16; ++j)
          if (i + j < n) acc = fmaf(m.weight[grp][i + j], t[j], acc);
      }
      acc += r;
      if (p.rmsnorm) p.yrow[(size_t)b * p.d + feat] = acc;
      else reinterpret_cast<unsigned short*>(p.y)[(size_t)b * p.d + feat] = to16(acc, p.bf16);
    }
    if (p.rmsnorm) {
      float sq = acc * acc;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, off);
      if (lane == 0) __stcg(p.ysq + (size_t)u * 4 + (gtid >> 5), sq);
    }
  }
  if (p.rmsnorm && !failed) {
    // every token's squares, in order, then the same thread's values again
    __syncthreads();
    if (tid == 0) {
      grid_arrive(&p.head->bar[3]);
      if (!grid_wait(&p.head->bar[3], gridDim.x + (p.missing == 3), bars)) dn_fail(bars, status);
      m.fail = dn_aborted(bars);
    }
    __syncthreads();
    for (int u = m.fail ? units : u0; u < units; u += ustep) {
      const int b = u / HT, feat = (u - b * HT) * kDnHalf + gtid;
      float t = 0.f;  // every warp alike
      for (int i = lane; i < 4 * HT; i += 32) t += __ldcg(p.ysq + (size_t)b * 4 * HT + i);
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) t += __shfl_xor_sync(0xffffffffu, t, off);
      const float scale = rsqrtf(t / (float)p.d + 1e-6f);
      if (feat < p.d) {
        const size_t at = (size_t)b * p.d + feat;
        reinterpret_cast<unsigned short*>(p.y)[at] = to16(p.yrow[at] * scale, p.bf16);
      }
    }
  }
  // The last CTA to leave clears the barriers for the next call; where a CTA gave up (counted in the upper half),
  // the counts that may have been left halfway, too.
  if (tid == 0) {
    const unsigned gave_up = dn_aborted(bars) ? 1u << 16 : 0u;
    unsigned old;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], %2;"
                 : "=r"(old)
                 : "l"(&p.head->bar[4]), "r"(1u + gave_up)
                 : "memory");
    if ((old & 0xffffu) == gridDim.x - 1) {
      for (int i = 0; i < 5; ++i) p.head->bar[i] = 0u;
      if ((old >> 16) + gave_up) {
        for (int i = 0; i < 64; ++i) p.head->tok[i] = 0u;
        for (int i = 0; i < kDnMaxCtas; ++i) p.head->cnt[i] = 0u;
      }
    }
  }
}

}  // namespace

size_t dense_layer_ws_bytes(int B, int d, int f, int E, int k, int ns, int sms) {
  return layer_plan(B, d, f, E, k, ns, sms, sizeof(LayerMisc), sizeof(DenseHead)).total;
}

cudaError_t launch_dense_layer(const DenseLayerCall& c, void* ws, int sms, int smem_optin, cudaStream_t st) {
  const LayerPlan& l = layer_plan(c.B, c.d, c.f, c.routed.E, c.k, c.shared.E, sms, sizeof(LayerMisc), sizeof(DenseHead));
  uint8_t* w8 = reinterpret_cast<uint8_t*>(ws);
  LayerMaps maps;
  cudaError_t e = cudaSuccess;
  auto set_maps = [&](const DenseExpertSet& s, CUtensorMap* g, CUtensorMap* u, CUtensorMap* d) {
    if (e == cudaSuccess)
      e = dense_map(g, s.gate_t, c.bf16, c.d, c.f, s.gate_rs, s.E, s.gate_rs * c.f, l.rows);
    if (e == cudaSuccess) e = dense_map(u, s.up_t, c.bf16, c.d, c.f, s.up_rs, s.E, s.up_rs * c.f, l.rows);
    if (e == cudaSuccess) e = dense_map(d, s.down, c.bf16, c.d, c.f, s.down_rs, s.E, s.down_rs * c.f, kDnChunk);
  };
  set_maps(c.routed, &maps.gate, &maps.up, &maps.down);
  if (c.shared.E > 0) set_maps(c.shared, &maps.sgate, &maps.sup, &maps.sdown);
  if (c.shared.E == 0) {
    maps.sgate = maps.gate;
    maps.sup = maps.up;
    maps.sdown = maps.down;
  }
  if (e == cudaSuccess) e = dense_map(&maps.x, c.x, c.bf16, c.d, c.B, c.d, 0, 0, 1);
  if (e == cudaSuccess) e = dense_map(&maps.h, w8 + l.h, c.bf16, c.f, (uint64_t)l.groups * 16, c.f, 0, 0, 16);
  if (e != cudaSuccess) return e;
  LayerArgs p;
  p.B = c.B;
  p.d = c.d;
  p.f = c.f;
  p.E = c.routed.E;
  p.k = c.k;
  p.ns = c.shared.E;
  p.renorm = c.renorm;
  p.rmsnorm = c.rmsnorm;
  p.bf16 = c.bf16;
  p.x = c.x;
  p.w_router = c.w_router;
  p.residual = c.residual;
  p.y = c.y;
  p.user_idx = c.user_idx;
  p.user_w = c.user_w;
  p.head = reinterpret_cast<DenseHead*>(ws);
  p.tries = c.tries ? c.tries : kWaitTries;
  p.missing = c.tries ? c.missing : -1;
  p.logits = reinterpret_cast<float*>(w8 + l.logits);
  p.top_idx = reinterpret_cast<int*>(w8 + l.top_idx);
  p.top_w = reinterpret_cast<float*>(w8 + l.top_w);
  p.h = reinterpret_cast<unsigned short*>(w8 + l.h);
  p.part = reinterpret_cast<float*>(w8 + l.part);
  p.ysum = reinterpret_cast<float*>(w8 + l.ysum);
  p.cut = (l.part - l.ysum) / 4;
  p.yrow = reinterpret_cast<float*>(w8 + l.yrow);
  p.ysq = reinterpret_cast<float*>(w8 + l.ysq);
  p.slots = l.groups * 8;
  p.rows = l.rows;
  p.early = l.early;
  p.slices = l.slices;
  p.block_rows = p.E % 8 && p.E >= 8 ? 3 : 0;
  p.block_vecs = p.E < 8 ? p.E : (p.E << p.block_rows) / 8;
  p.blocks = kDnThreads / p.block_vecs;
  p.sum_step = (p.E < 16 ? 16 : kDnThreads / p.E) * p.E;
  p.a_bytes = layer_a_bytes(l.rows, l.wide);
  p.stage_bytes = p.a_bytes + (c.B + 7) / 8 * 16 * 128;
  const int fixed = 1024 + (int)sizeof(LayerMisc) + p.slots;
  int S = (smem_optin - fixed) / p.stage_bytes;
  p.stages = S > kDnMaxStages ? kDnMaxStages : S;
  if (p.stages < 3 || l.grid < c.B) return cudaErrorInvalidValue;  // routing: a CTA for every token
  const size_t smem = fixed + (size_t)p.stages * p.stage_bytes;
  static std::atomic<uint64_t> allowed[2];
  const auto kernel = l.wide == 2 ? dense_layer_kernel<2> : dense_layer_kernel<1>;
  e = allow_shared(kernel, allowed[l.wide - 1], smem_optin);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(l.grid);
  cfg.blockDim = dim3(kDnThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeCooperative;
  attr[0].val.cooperative = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, maps, p);
}

}  // namespace sesg
