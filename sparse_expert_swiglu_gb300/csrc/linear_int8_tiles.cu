// The products of linear_int8.cu for more than a few tokens, on the tensor cores.
//
// Sums are exact integers: the operands are integers of 8 bits, which fp16 holds, their products are no larger than 2^14 and
// 1024 of them than 2^24, up to which an fp32 accumulator holds every integer.  (This chip's tensor cores have next to no
// rate for 8-bit integers: mma.sync takes as long as dp4a.)  So a tile's k goes in rounds of 1024; two sets of accumulators take
// turns, and the epilogue's warps add the rounds up as 32-bit integers in registers under the next round's products.
//
// The features lie on the 128 TMEM lanes (with w_mul 64 of each matrix), the tokens on the columns.  w comes from HBM in 8 bits;
// eight warps turn 64 k of 128 rows at a time into fp16 on the way from shared memory to TMEM, where the products read them as
// operand A: the conversion costs shared memory one read of a byte a weight, and no second copy of w exists anywhere.  (In shared
// memory the fp16 tile would be written and read again, 6 bytes a weight.)  The tokens, few beside w or used by many tiles,
// have been made fp16 integers by the kernel before (quantize.cu).  w's copies start before that kernel is done.
//
// Where there are fewer tiles than SMs, a cluster's CTAs share a tile along k and join their sums in shared memory; with many
// tokens CTA pairs run one product, so that each fetches half of the tokens.  int8_plan chooses.
//
// Measured: 2048 tokens of 2 x 14336 x 4096 326 us (1.48 PFLOP/s; tensor cores busy 63 %: a stage of a pair takes 5.6 clocks
// for each token, of which the products are 4, as shared memory serves the loads, the conversion and the products); 48 of 2 x
// 16384 x 6144 42.3 us (4.8 TB/s); 16 of 4096 x 4096 9.4 us and 64 of them 11.4, 1.5 of that the tokens' kernel and 2.2 the
// join.  What a short call feels beside its bytes is code: integer divisions (100 to 200 clocks each, some 2.5 us a call before
// they went), barriers, lines of code that no call before has fetched.
#include "activate.cuh"
#include "dense.cuh"
#include "dense_params.cuh"
#include "int8.cuh"
#include "int8_params.cuh"
#include "int8_plan.h"

#include <type_traits>

namespace sesg {

namespace {

struct TileArgs {
  int M, N, bf16, act, out_f32;
  int MT, NT, T, KC, S;
  int rows;                // features of a CTA's tile: up to 128, with w_mul 64
  int stages, slots;
  int stream;              // w is read once
  const float* x_scale;    // with room for whole blocks of 16 tokens
  const float *w_scale, *w_mul_scale;
  const void *bias, *bias_mul, *residual;
  void* y;
  DenseHead* head;
  uint32_t tries;          // rounds of a wait
  int missing;             // diagnostics: the first CTA's stages wait for an arrival that does not come
};

struct alignas(16) TileBars {
  DenseBars d;
  uint64_t afull[kI8MaxSlots];   // a slot has its fp16 weights
  uint64_t aempty[kI8MaxSlots];  // its products are done
};
static_assert(sizeof(TileBars) % 16 == 0, "what follows is read 16 bytes at a time");

// D += A B with A in TMEM, fp16 operands
template <bool PAIR>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t desc, uint32_t add) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(desc), "r"(add)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(desc), "r"(add)
        : "memory");
}

// 32 columns of this warp's 32 lanes
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,"
      "%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]),
      "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}

// 16 bytes into a CTA of the cluster, counted on that CTA's barrier
__device__ __forceinline__ void peer_store(uint32_t to, const int* v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(bar)
               : "memory");
}

__device__ __forceinline__ void tile_of(int t, int T, int MT, int& ft, int& mt) {
  if (MT == 1) {
    ft = t;
    mt = 0;
    return;
  }
  const int block = T / MT * kTogether, b = t / block, r = t - b * block;
  const int here = MT - b * kTogether < kTogether ? MT - b * kTogether : kTogether;
  ft = r / here;
  mt = b * kTogether + r - ft * here;
}

// One feature's scale and bias in one matrix.
struct Feature {
  float scale, bias;
  __device__ Feature(float s, float b) : scale(s), bias(b) {}
  __device__ Feature(const TileArgs& p, bool mul, int feat, bool on) {
    scale = on ? (mul ? p.w_mul_scale : p.w_scale)[feat] : 0.f;
    const void* b = mul ? p.bias_mul : p.bias;
    bias = on && b ? ld16(b, feat, p.bf16) : 0.f;
  }
};

// The scales of W tokens (a multiple of 4).
template <int W>
__device__ __forceinline__ void token_scales(const float* from, float (&xs)[W]) {
#pragma unroll
  for (int i = 0; i < W; i += 4) {
    const float4 t = *reinterpret_cast<const float4*>(from + i);
    xs[i] = t.x;
    xs[i + 1] = t.y;
    xs[i + 2] = t.z;
    xs[i + 3] = t.w;
  }
}

// The residual of W tokens from tok of one feature; n of them exist.
template <int W>
__device__ __forceinline__ void tile_residual(const TileArgs& p, int feat, int tok, int n, unsigned short (&r)[W]) {
  if (!p.residual) return;
  const unsigned short* from = reinterpret_cast<const unsigned short*>(p.residual) + (size_t)tok * p.N + feat;
#pragma unroll
  for (int i = 0; i < W; ++i) r[i] = i < n ? from[(size_t)i * p.N] : (unsigned short)0;
}

// Residual and store of W tokens' values of one feature; token i at offset at + i * N.
template <int W, bool FULL>
__device__ __forceinline__ void tile_write(const TileArgs& p, size_t at, int n, float (&v)[W], const unsigned short (&r)[W]) {
  if (p.residual) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = __fadd_rn(v[i], from16(r[i], p.bf16));
  }
  if (p.out_f32) {
    float* y = reinterpret_cast<float*>(p.y) + at;
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (FULL || i < n) y[(size_t)i * p.N] = v[i];
    return;
  }
  unsigned short* y = reinterpret_cast<unsigned short*>(p.y) + at;
  unsigned short t[W];
  if (p.bf16) {
#pragma unroll
    for (int i = 0; i < W; ++i) t[i] = to16(v[i], 1);
  } else {
#pragma unroll
    for (int i = 0; i < W; ++i) t[i] = to16(v[i], 0);
  }
#pragma unroll
  for (int i = 0; i < W; ++i)
    if (FULL || i < n) y[(size_t)i * p.N] = t[i];
}

// Activation, product with m (with w_mul), residual and store of W tokens from tok of one feature; n of them exist.
template <int W, bool GATED>
__device__ __forceinline__ void tile_store(const TileArgs& p, int feat, int tok, int n, float (&v)[W], const float* m,
                                           const unsigned short (&r)[W]) {
  activate<W, true>(v, p.act);
  if (GATED) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] = __fmul_rn(v[i], m[i]);
  }
  const size_t at = (size_t)tok * p.N + feat;
  if (W >= 8 && n >= W) tile_write<W, true>(p, at, n, v, r);
  else tile_write<W, false>(p, at, n, v, r);
}

// Arrives at a barrier of the pair's first CTA.  What it orders lies in TMEM alone, behind tcgen05's own fences (tokens in shared
// memory count on a barrier there); the release over the cluster of peer_arrive would wait 1200 clocks for the thread's
// other stores.
__device__ __forceinline__ void pair_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// The two halves of cluster_sync_all.
__device__ __forceinline__ void cluster_leave() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_left() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// The sums of a tile that a cluster's CTAs share: each finishes its part of them.  A unit is 16 of every 32 tokens of 32
// features, 8 of a tile or 4 with w_mul, for S CTAs; 8 CTAs take every other group of 4 tokens of a unit of 4.  A cell is one
// lane's 4 tokens of 32 features, 512 bytes, at [rank][matrix][cell of the owner's][lane], in the owner's stages: from behind
// the last one that it uses on, whose products are done before all others'.
template <bool GATED>
struct Cells {
  static constexpr int kLogUnits = GATED ? 2 : 3;
  int g4, log_per, count;  // groups of 4 tokens of a unit; a CTA's units (2 to that power) and cells
  bool odd;                // owners by groups
  __device__ Cells(int NT, int log_s) : g4((NT + 31) / 32 * 4), odd(log_s > kLogUnits) {
    log_per = odd ? 0 : kLogUnits - log_s;
    count = odd ? g4 / 2 : g4 << log_per;
  }
  __device__ int owner(int unit, int g) const { return odd ? 2 * unit + (g & 1) : unit >> log_per; }
  __device__ int first(int unit) const { return odd ? 0 : (unit & ((1 << log_per) - 1)) * g4; }  // cell of its owner's
  // a CTA's cells, by a step below or at g4 * 8: the unit and the group of the one after
  __device__ void start(int rank, int cell, int& unit, int& g) const {
    unit = odd ? rank >> 1 : rank << log_per;
    g = odd ? rank & 1 : 0;
    step(cell, unit, g);
  }
  __device__ void step(int by, int& unit, int& g) const {
    g += odd ? 2 * by : by;
    for (; g >= g4 && !odd; g -= g4) ++unit;
  }
  static __device__ int token(int unit, int g) { return 32 * (g >> 2) + 16 * (unit & 1) + 4 * (g & 3); }  // the first
  __device__ int bytes(int S) const { return S * (GATED ? 2 : 1) * count * 512; }
};

// PAIR: CTA pairs, whose tile has 256 features, 128 in each CTA, which keeps half of the tokens.  SHARED: clusters share a
// tile along k, one tile for each.  GATED: with w_mul; 64 features of w, then the same ones of w_mul.  TB: blocks of 16 columns
// that an epilogue warp adds up.  KS: 64 k in a slot.
template <bool PAIR, bool SHARED, bool GATED, int TB, int KS>
__global__ void __launch_bounds__(kI8Threads, 1)
int8_tile_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mw2,
                 const __grid_constant__ CUtensorMap mx, const TileArgs p) {
  extern __shared__ uint8_t raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  constexpr int P = PAIR ? 2 : 1;
  // With up to 64 tokens there are no fewer slots than stages: a slot is free when its stage is.
  constexpr bool kSlotWaits = TB > 2;
  const int feats = p.rows;
  constexpr uint32_t kW = 128 * kI8Chunk;  // bytes of a stage's rows of w
  const int NT = p.NT, toks = NT / P, ns = p.stages;
  const uint32_t tok_bytes = toks * 128, stage_bytes = kW + 2 * tok_bytes;
  const int load_rows = p.N < feats ? p.N : feats, load_toks = p.M < toks ? p.M : toks;  // boxes no higher than the operands
  TileBars* tb = reinterpret_cast<TileBars*>(ring + (size_t)ns * stage_bytes);
  float* halves = reinterpret_cast<float*>(tb + 1) + kI8Cols / 2 * 8;  // GATED: what pairs of epilogue warps exchange
  DenseBars* bars = &tb->d;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int S = SHARED ? p.S : 1;
  const int crank = PAIR || SHARED ? (int)cluster_rank() : 0, half_of = PAIR ? crank & 1 : 0, lead = crank - half_of;
  const int rank = SHARED ? crank / P : 0;
  // what a stage's barrier counts: of a pair, the first CTA's both CTAs' tokens, the second's its weights alone
  const uint32_t load_bytes = (GATED ? 2 : 1) * load_rows * kI8Chunk + (PAIR ? 2 - 2 * half_of : 1) * 2 * load_toks * 128;
  const int log_s = SHARED ? __ffs(S) - 1 : 0;  // (divisions take 100 to 200 clocks each, which a call of few tokens feels)
  const int first = blockIdx.x >> (P - 1 + log_s), step = gridDim.x >> (P - 1 + log_s);
  const int kc0 = p.KC * rank >> log_s, kc1 = p.KC * (rank + 1) >> log_s;
  const int tiles = first < p.T ? (p.T - first + step - 1) / step : 0;
  int* status = &p.head->ctrl.status;
  const uint32_t ring_at = smem_addr(ring);

  if (tid == 0) {
    dn_init_bars(bars, p.tries, P * 8, 1 + (p.missing && blockIdx.x == 0));
    for (int i = 0; i < kI8MaxSlots; ++i) {
      mbar_init(&tb->afull[i], 4 * P);
      mbar_init(&tb->aempty[i], 1);
    }
    mbar_init(&bars->xready, S);
    mbar_init(&bars->xfull, 1);
    fence_barrier_init();
    tma_prefetch_map(&mw);
    tma_prefetch_map(&mx);
    if (GATED) tma_prefetch_map(&mw2);
  }
  if (warp == 2) {
    if (PAIR) tmem_alloc_pair(&bars->tmem, 512);
    else tmem_alloc(&bars->tmem, 512);
  }
  tc_before_sync();
  __syncthreads();
  if (PAIR || SHARED) cluster_sync_all();  // the barriers are there before any CTA of the cluster uses them
  tc_after_sync();
  const uint32_t tmem = bars->tmem;
  const uint32_t slots_at = tmem + 2 * NT;
  // The kernel before is the tokens' (quantize.cu): it started its dependents behind its own wait, so that everything
  // before it is done, and only what it writes, tokens and scales, has to be waited for.
  griddep_launch_dependents();

  // (setmaxnreg is one instruction for all warps of a warpgroup: four from a multiple of four on.)
  const Cells<GATED> cells(NT, log_s);
  bool left = false;  // this thread has told the cluster that it is done with it
  if (warp < 4) {
    if constexpr (TB >= 4) fewer_registers<kI8RegsIssue>();
    if (SHARED && warp == 3) {
      // what comes into this CTA from all of the cluster (a store that were counted before this would be as well)
      int ft, mt, there = 0, unit, g;
      tile_of(first, p.T, p.MT, ft, mt);
      cells.start(rank, lane, unit, g);
      for (int i = lane; i < cells.count; i += 32, cells.step(32, unit, g)) there += mt * NT + cells.token(unit, g) < p.M;
      there = __reduce_add_sync(0xffffffffu, there);
      if (lane == 0) mbar_arrive_expect_tx(&bars->xfull, there * 512 * S * (GATED ? 2 : 1));
    }
    if (warp == 0) {
      if (elect_one()) {
        const uint64_t pw = p.stream ? policy_evict_first() : policy_evict_normal();
        const uint64_t px = policy_evict_normal();
        int st = 0, issued = 0;
        uint32_t ph = 0;
        bool ok = true;
        auto weights = [&](int s, int kc, int ft) {
          const int f0 = (ft * P + half_of) * feats;
          mbar_arrive_expect_tx(&bars->full[s], load_bytes);
          ++issued;
          const uint32_t a = ring_at + s * stage_bytes;
          tma_2d(a, &mw, kc * kI8Chunk, f0, &bars->full[s], pw);
          if (GATED) tma_2d(a + kW / 2, &mw2, kc * kI8Chunk, f0, &bars->full[s], pw);
        };
        // A pair's tokens count on the first CTA's barrier: its converting warps wait for that, and the products, which read
        // both CTAs' tokens, for those warps.
        const uint32_t full_at = PAIR ? peer_addr(smem_addr(&bars->full[0]), lead) : 0;
        auto tokens = [&](int s, int kc, int mt) {
          const int m0 = mt * NT + half_of * toks;
          const uint32_t b = ring_at + s * stage_bytes + kW;
          if constexpr (PAIR) {
            tma_2d_pair(b, &mx, kc * kI8Chunk, m0, full_at + s * 8, px);
            tma_2d_pair(b + tok_bytes, &mx, kc * kI8Chunk + 64, m0, full_at + s * 8, px);
          } else {
            tma_2d(b, &mx, kc * kI8Chunk, m0, &bars->full[s], px);
            tma_2d(b + tok_bytes, &mx, kc * kI8Chunk + 64, m0, &bars->full[s], px);
          }
        };
        int ahead = 0;  // stages of the first tile whose weights are under way before the tokens can be
        if (first < p.T) {
          int ft, mt;
          tile_of(first, p.T, p.MT, ft, mt);
          for (; ahead < ns && kc0 + ahead < kc1; ++ahead) weights(ahead, kc0 + ahead, ft);
        }
        griddep_wait();
        for (int t = first; ok && t < p.T; t += step) {
          int ft, mt;
          tile_of(t, p.T, p.MT, ft, mt);
          for (int kc = kc0; kc < kc1; ++kc) {
            if (ahead > 0) {
              --ahead;
            } else {
              if (!dn_wait(&bars->empty[st], ph ^ 1, bars)) {
                dn_fail(bars, status);
                ok = false;
                break;
              }
              weights(st, kc, ft);
            }
            tokens(st, kc, mt);
            if (++st == ns) {
              st = 0;
              ph ^= 1;
            }
          }
        }
        if (SHARED && ok) {
          // The stages behind the last one are free when their products are done (this thread has seen every phase of
          // theirs but the last end): the cluster may store there, under the products of the others.
          const int count = kc1 - kc0;
          for (int at = 0, c = count - ns; ok && at < cells.bytes(S); at += stage_bytes, ++c)
            ok = c < 0 || dn_wait(&bars->empty[c % ns], c / ns & 1, bars);
          if (!ok) dn_fail(bars, status);
          for (int i = 0; ok && i < S; ++i) peer_arrive(peer_addr(smem_addr(&bars->xready), P * i + half_of));
        }
        // No copy of this CTA is in flight when it ends: the last stages have come.  A pair has used every copy when its
        // epilogues are done, and one that gave up waits at its end (else for copies that the other CTA may not have issued).
        const int n = PAIR ? 0 : issued < ns ? issued : ns;
        for (int i = 0; i < n; ++i) {
          if (--st < 0) {
            st = ns - 1;
            ph ^= 1;
          }
          dn_drain(&bars->full[st], ph, p.tries);
        }
      }
    } else if (warp == 1) {
      if (crank == lead && elect_one()) {
        const uint32_t desc = mma_desc(NT, 0, 0, P * 128);
        auto commit = [&](uint64_t* bar) {
          if constexpr (PAIR) mma_commit_pair(bar, lead);
          else mma_commit(bar);
        };
        int st = 0, buf = 0, slot = 0;
        uint32_t tph = 0, sph = 0;
        bool ok = true, open = false;
        for (int t = 0; ok && t < tiles; ++t) {
          for (int kr = kc0, end; ok && kr < kc1; kr = end) {
            end = kr + kI8Round < kc1 ? kr + kI8Round : kc1;
            if (!(PAIR ? cluster_wait(&bars->tempty[buf], tph ^ 1, bars) : dn_wait(&bars->tempty[buf], tph ^ 1, bars))) {
              dn_fail(bars, status);
              ok = false;
              break;
            }
            tc_after_sync();
            const uint32_t d = tmem + buf * NT;
            // (One way back for each stage: a jump costs the issuing thread some 200 to 400 clocks beside 19 other warps.)
#pragma unroll 2
            for (int kc = kr; kc < end; ++kc) {
              const uint64_t bd = smem_desc(ring_at + st * stage_bytes + kW, 16);
#pragma unroll
              for (int hk = 0; hk < 2; hk += KS) {
                if (!(PAIR ? cluster_wait(&tb->afull[slot], sph, bars) : dn_wait(&tb->afull[slot], sph, bars))) {
                  ok = false;
                  break;
                }
                tc_after_sync();
                const uint32_t a = slots_at + slot * 32 * KS;
#pragma unroll
                for (int ks = 0; ks < 4 * KS; ++ks)
                  mma_ts<PAIR>(d, a + ks * 8, bd + (hk || ks >= 4 ? tok_bytes >> 4 : 0) + (ks & 3) * 2, desc,
                               hk > 0 || ks > 0 || kc > kr);
                if (kSlotWaits) commit(&tb->aempty[slot]);
                open = true;
                const bool wrap = ++slot == p.slots;
                slot = wrap ? 0 : slot;
                sph ^= wrap;
              }
              if (!ok) break;
              commit(&bars->empty[st]);
              st = st + 1 == ns ? 0 : st + 1;
            }
            if (!ok) {
              dn_fail(bars, status);
              break;
            }
            commit(&bars->tfull[buf]);
            if (++buf == 2) {
              buf = 0;
              tph ^= 1;
            }
          }
        }
        if (open) {  // every product is done before TMEM is given back
          commit(&bars->drain);
          dn_drain(&bars->drain, 0, kWaitTries);
        }
      }
    }
  } else if (warp < 12) {
    // Every other stage, of the 32 rows whose TMEM lanes this warp may write.  The number of stages is even, so that a stage is
    // always the same warps': a wait by parity tells a phase only from the one before it, which its warps must have seen end.
    // (With seven, warps that ran ahead took a stage that the others had not seen loaded for their own next one: 3 of 80000
    // calls of 4 tokens by 32000 x 4096 came to a stop.)  A slot's last use but one lies four stages back or more, and these
    // warps have waited for the products of one four stages back when they took their stage before this.
    if constexpr (TB >= 4) fewer_registers<kI8RegsConvert>();
    const int q = warp & 3, set = (warp - 4) >> 2, row = q * 32 + lane;
    const uint32_t lanes = slots_at + ((uint32_t)(q * 32) << 16);
    const int total = tiles * (kc1 - kc0);
    int st = set, slot = set * (2 / KS);
    uint32_t ph = 0, sph = 0;
    bool ok = true;
#pragma unroll 1
    for (int it = set; ok && it < total; it += 2) {
      ok = dn_wait(&bars->full[st], ph, bars);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {
        if (lane == 0) dn_fail(bars, status);
        break;
      }
      const uint32_t from = ring_at + st * stage_bytes + row * 128;
      // (Both halves are read first where there are registers for them.)
      constexpr int H = TB > 2 ? 1 : 2;
      uint4 w[4 * H];
      auto read = [&](int hk, int h) {
#pragma unroll
        for (int c = 0; c < 4; ++c) w[4 * h + c] = ld_shared_v4(from + (((4 * hk + c) ^ (row & 7)) << 4));
      };
      read(0, 0);
      if (H == 2) read(1, 1);
      if (!kSlotWaits) tc_after_sync();
#pragma unroll
      for (int hk = 0; hk < 2; ++hk) {
        if (H == 1 && hk == 1) read(1, 0);
        uint32_t v[32];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4& t = w[H == 2 ? 4 * hk + c : c];
          to_f16(t.x, v[8 * c], v[8 * c + 1]);
          to_f16(t.y, v[8 * c + 2], v[8 * c + 3]);
          to_f16(t.z, v[8 * c + 4], v[8 * c + 5]);
          to_f16(t.w, v[8 * c + 6], v[8 * c + 7]);
        }
        if (kSlotWaits && (KS == 1 || hk == 0)) {
          ok = PAIR ? cluster_wait(&tb->aempty[slot], sph ^ 1, bars) : dn_wait(&tb->aempty[slot], sph ^ 1, bars);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          tc_after_sync();
        }
        tmem_st32(lanes + (slot * KS + (KS == 2 ? hk : 0)) * 32, v);
        if (hk == 1 || KS == 1) {
          tmem_stored();
          tc_before_sync();
          __syncwarp();
          if (lane == 0) {
            // (the first CTA's arrival also hands on the tokens of both that its stage's barrier has counted)
            if (PAIR && half_of) pair_arrive(peer_addr(smem_addr(&tb->afull[slot]), lead));
            else mbar_arrive(&tb->afull[slot]);
          }
        }
        if (KS == 1 && hk == 0) {
          const bool wrap = ++slot == p.slots;
          slot = wrap ? 0 : slot;
          sph ^= wrap;
        }
      }
      if (!ok && lane == 0) dn_fail(bars, status);
      slot += KS == 1 ? 3 : 2;
      const bool wrap = slot >= p.slots;
      slot -= wrap ? p.slots : 0;
      sph ^= wrap;
      st += 2;
      const bool turn = st >= ns;
      st -= turn ? ns : 0;
      ph ^= turn;
    }
  } else {
    // Lanes 32 (warp % 4) ... are this warp's.  Of the two warps that have them, each takes every other 16 tokens.
    if constexpr (TB >= 4) more_registers<kI8RegsEpilogue>();
    const int q = warp & 3, half = (warp - 12) >> 2;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16);
    int buf = 0;
    uint32_t tph = 0;
    griddep_wait();  // the tokens' scales
    for (int t = first; t < p.T; t += step) {
      int ft, mt;
      tile_of(t, p.T, p.MT, ft, mt);
      const int m0 = mt * NT, nt = p.M - m0 < NT ? p.M - m0 : NT, f0 = (ft * P + half_of) * feats;
      // this lane's feature (of the one or the other matrix), and in shared memory this half's tokens' scales: both are under
      // way while the sums are
      const int mul = GATED ? q >> 1 : 0, local = (GATED ? q & 1 : q) * 32 + lane, feat = f0 + local;
      const bool on = local < feats && feat < p.N;
      float* scales = reinterpret_cast<float*>(tb + 1) + (warp - 12) * (kI8Cols / 2);
      Feature f = {0.f, 0.f};
      ScaleRange range;
      if (!SHARED) {
        f = Feature(p, mul, feat, on);
        __syncwarp();
        for (int i = lane; 32 * (i >> 4) + 16 * half < nt; i += 32) {
          const int tok = 32 * (i >> 4) + 16 * half + (i & 15);
          const float s = p.x_scale[m0 + tok];
          scales[i] = s;
          if (tok < nt) range.add(s);
        }
        range.join();
        __syncwarp();
      }
      // Where a cluster's sums go: those of even and of odd groups of 4 tokens.
      const int ring_bytes = ns * (int)stage_bytes;
      auto place = [&](int r) {  // CTA r's begin
        return ((p.KC * (r + 1) >> log_s) - (p.KC * r >> log_s)) % ns * (int)stage_bytes;
      };
      auto wrap = [&](int at) { return at < ring_bytes ? at : at - ring_bytes; };
      int to[2] = {0, 0}, cta[2] = {0, 0}, from = 0;
      if constexpr (SHARED) {
        const int unit = GATED ? (q & 1) * 2 + half : 2 * q + half;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int r = cells.owner(unit, i);
          to[i] = place(r) + ((rank * (GATED ? 2 : 1) + mul) * cells.count + cells.first(unit)) * 512 + lane * 16;
          cta[i] = P * r + half_of;
        }
        from = place(rank) + lane * 16;
      }
      bool ok = true;
      auto release = [&] {  // this set of accumulators has been read
        tc_before_sync();
        __syncwarp();
        if (lane == 0) {
          if (PAIR) pair_arrive(peer_addr(smem_addr(&bars->tempty[buf]), lead));
          else mbar_arrive(&bars->tempty[buf]);
        }
        if (++buf == 2) {
          buf = 0;
          tph ^= 1;
        }
      };
      auto sums_there = [&] {
        ok = dn_wait(&bars->tfull[buf], tph, bars);
        if (!ok) dn_fail(bars, status);
        ok = !dn_any(1, 256, !ok);  // one decision for the warps
        tc_after_sync();
        return ok;
      };
      // Rounds are added up in registers, which frees TMEM for the next tile's products before this one's epilogue.
      int acc[TB][16];
#pragma unroll
      for (int b = 0; b < TB; ++b)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[b][i] = 0;
#pragma unroll 1
      for (int kr = kc0; kr < kc1; kr += kI8Round) {
        if (!sums_there()) break;
#pragma unroll
        for (int b = 0; b < TB; ++b) {
          const int n0 = 32 * b + 16 * half;
          if (n0 >= NT) continue;  // the same for the whole warp
          float v[16];
          tmem_ld(lanes + buf * NT + n0, v);
          tmem_wait(v);
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[b][i] += __float2int_rn(v[i]);
        }
        release();
      }
      if (!ok) break;
      // the next sums to acc[0]: the epilogue's code is there once
      auto turn_blocks = [&](auto by) {
        constexpr int W = decltype(by)::value;
#pragma unroll
        for (int i = 0; i + W < TB * 16; ++i) acc[i / 16][i % 16] = acc[(i + W) / 16][(i + W) % 16];
      };
      // Two copies, so that a decision for each tile is enough (one for each value costs 2048 tokens of 14336 x 4096 168 us for
      // 158, one for each 16 160; gated, 2 x 14336 x 4096, both 337 to 349 for 320 and this 325).
      auto finish = [&](auto any) {
        constexpr bool ODD = decltype(any)::value;
        auto value = [&](int sum, float x_scale) {
          return ODD ? int8_value(sum, x_scale, f.scale, f.bias)
                     : int8_scaled((float)sum, __fmul_rn(x_scale, f.scale), f.bias);
        };
        if constexpr (!GATED) {
          // W tokens at a time: a short call pays for every line of code that it fetches
          constexpr int W = TB <= 2 || ODD ? 8 : 16;
          for (int n0 = 16 * half; n0 < nt; n0 += 32)
#pragma unroll 1
            for (int i = n0; i < n0 + 16; i += W) {
              unsigned short r[W];
              float xs[W], v[W];
              if (on) tile_residual(p, feat, m0 + i, nt - i, r);
              token_scales(scales + (n0 >> 5) * 16 + (i & 15), xs);
#pragma unroll
              for (int j = 0; j < W; ++j) v[j] = value(acc[0][j], xs[j]);
              if (on) tile_store<W, false>(p, feat, m0 + i, nt - i, v, nullptr, r);
              turn_blocks(std::integral_constant<int, W>());
            }
        } else {
          // Warps q and q + 2 have the two matrices' sums of the same features: of 16 tokens the first finishes eight and
          // the second eight, and each gives the other what it lacks.
          const int pair = (q & 1) * 2 + half;
          int turn = 0;
#pragma unroll 1
          for (int n0 = 16 * half; n0 < nt; n0 += 32) {
            float xs[16];
            unsigned short r[8];
            const int tok = n0 + 8 * mul;  // the eight of this warp
            if (on) tile_residual(p, feat, m0 + tok, nt - tok, r);
            token_scales(scales + (n0 >> 5) * 16, xs);
            float* give = halves + ((turn * 4 + pair) * 2 + mul) * 256 + lane;
            const float* take = halves + ((turn * 4 + pair) * 2 + (mul ^ 1)) * 256 + lane;
            float v[8], m[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float a = value(acc[0][j], xs[j]), b = value(acc[0][8 + j], xs[8 + j]);
              v[j] = mul ? b : a;
              give[32 * j] = mul ? a : b;
            }
            named_barrier(2 + pair, 64);  // (the next turn's writes go to the other buffer)
            turn ^= 1;
#pragma unroll
            for (int j = 0; j < 8; ++j) m[j] = take[32 * j];
            if (mul) {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const float a = m[j];
                m[j] = v[j];
                v[j] = a;
              }
            }
            if (on) tile_store<8, true>(p, feat, m0 + tok, nt - tok, v, m, r);
            turn_blocks(std::integral_constant<int, 16>());
          }
        }
      };
      if constexpr (!SHARED) {
        // whether a product of the warp's scales may leave fp32's normal range
        if (__any_sync(0xffffffffu, range.odd(f.scale))) finish(std::true_type());
        else finish(std::false_type());
      } else {
        int cell_unit, cell_g;
        cells.start(rank, warp - 12, cell_unit, cell_g);
        ok = cluster_wait(&bars->xready, 0, bars);
        if (!ok) dn_fail(bars, status);
        if (dn_any(1, 256, !ok)) break;
#pragma unroll 1
        for (int n0 = 16 * half; n0 < nt; n0 += 32) {
#pragma unroll
          for (int h = 0; h < 4; ++h)
            if (n0 + 4 * h < nt)
              peer_store(peer_addr(ring_at + wrap(to[h & 1] + (((n0 >> 5) * 4 + h) >> cells.odd) * 512), cta[h & 1]),
                         &acc[0][4 * h], peer_addr(smem_addr(&bars->xfull), cta[h & 1]));
          turn_blocks(std::integral_constant<int, 16>());
        }
        ok = cluster_wait(&bars->xfull, 0, bars);
        if (!ok) dn_fail(bars, status);
        if (dn_any(1, 256, !ok)) break;
        __syncwarp();
        cluster_leave();  // (nothing comes into this CTA any more, and nothing leaves it)
        left = true;
        for (int cell = warp - 12; cell < cells.count; cell += 8, cells.step(8, cell_unit, cell_g)) {
          const int tok = cells.token(cell_unit, cell_g), at = (cell_unit >> 1) * 32 + lane, feat = f0 + at;
          if (tok >= nt || at >= feats || feat >= p.N) continue;
          float xs[4];
          unsigned short r[4];
          tile_residual(p, feat, m0 + tok, nt - tok, r);
          token_scales(p.x_scale + m0 + tok, xs);
          float v[2][4];
#pragma unroll
          for (int m = 0; m < (GATED ? 2 : 1); ++m) {
            const Feature fm(p, m, feat, true);
            int a[4] = {0, 0, 0, 0};
            for (int s = 0; s < S; ++s) {
              const int at_s = wrap(from + ((s * (GATED ? 2 : 1) + m) * cells.count + cell) * 512);
              const int4 x = *reinterpret_cast<const int4*>(ring + at_s);
              a[0] += x.x;
              a[1] += x.y;
              a[2] += x.z;
              a[3] += x.w;
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) v[m][j] = int8_value(a[j], xs[j], fm.scale, fm.bias);
          }
          tile_store<4, GATED>(p, feat, m0 + tok, nt - tok, v[0], v[1], r);
        }
      }
    }
  }
  __syncwarp();
  tc_before_sync();
  if (PAIR || SHARED) {
    // no CTA ends while another may store into it or read its stages
    if (!left) cluster_leave();
    cluster_left();
    if (dn_aborted(bars)) dn_settle();  // stores that this CTA did not wait for
  } else {
    __syncthreads();
  }
  tc_after_sync();
  if (warp == 2) {
    if (PAIR) tmem_free_pair(tmem, 512);
    else tmem_free(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_int8_tiles(const LinearInt8Call& c, const void* tokens, const float* scales, void* ws, int sms,
                              int smem_optin, cudaStream_t st) {
  const bool gated = c.w_mul != nullptr;
  const int room = smem_optin - 1024 - (int)sizeof(TileBars) - int8_extra_bytes(gated);
  const Int8Plan& l = int8_plan(c.M, c.N, c.K, gated, sms, room);
  if (!l.S) return cudaErrorInvalidValue;
  CUtensorMap mw, mw2, mx;
  const uint32_t rows = c.N < l.rows ? c.N : l.rows, toks = c.M < l.NT / l.P ? c.M : l.NT / l.P;
  cudaError_t e = int8_map(&mw, c.w, c.K, c.N, rows);
  if (e != cudaSuccess) return e;
  mw2 = mw;
  if (gated) e = int8_map(&mw2, c.w_mul, c.K, c.N, rows);
  if (e == cudaSuccess) e = dense_map(&mx, tokens, 0, c.K, c.M, c.K, 0, 0, toks);
  if (e != cudaSuccess) return e;
  TileArgs p;
  p.M = c.M;
  p.N = c.N;
  p.bf16 = c.bf16;
  p.act = c.act;
  p.out_f32 = c.out_f32;
  p.MT = l.MT;
  p.NT = l.NT;
  p.T = l.T;
  p.KC = (c.K + kI8Chunk - 1) / kI8Chunk;
  p.S = l.S;
  p.rows = l.rows;
  p.stages = l.stages;
  p.slots = l.slots;
  p.stream = l.MT == 1;
  p.x_scale = scales;
  p.w_scale = c.w_scale;
  p.w_mul_scale = c.w_mul_scale;
  p.bias = c.bias;
  p.bias_mul = c.bias_mul;
  p.residual = c.residual;
  p.y = c.y;
  p.head = reinterpret_cast<DenseHead*>(ws);
  p.tries = c.tries ? c.tries : kWaitTries;
  p.missing = c.tries > 0;
  using Kernel = decltype(&int8_tile_kernel<false, false, false, 1, 2>);
  static constexpr Kernel kernels[32] = {
      int8_tile_kernel<false, false, false, 1, 2>, int8_tile_kernel<false, false, false, 2, 2>,
      int8_tile_kernel<false, false, false, 4, 2>, int8_tile_kernel<false, false, false, 6, 1>,
      int8_tile_kernel<false, false, true, 1, 2>, int8_tile_kernel<false, false, true, 2, 2>,
      int8_tile_kernel<false, false, true, 4, 2>, int8_tile_kernel<false, false, true, 6, 1>,
      int8_tile_kernel<false, true, false, 1, 2>, int8_tile_kernel<false, true, false, 2, 2>,
      int8_tile_kernel<false, true, false, 4, 2>, int8_tile_kernel<false, true, false, 6, 1>,
      int8_tile_kernel<false, true, true, 1, 2>, int8_tile_kernel<false, true, true, 2, 2>,
      int8_tile_kernel<false, true, true, 4, 2>, int8_tile_kernel<false, true, true, 6, 1>,
      nullptr, nullptr, int8_tile_kernel<true, false, false, 4, 2>, int8_tile_kernel<true, false, false, 6, 1>,
      nullptr, nullptr, int8_tile_kernel<true, false, true, 4, 2>, int8_tile_kernel<true, false, true, 6, 1>,
      nullptr, nullptr, int8_tile_kernel<true, true, false, 4, 2>, int8_tile_kernel<true, true, false, 6, 1>,
      nullptr, nullptr, int8_tile_kernel<true, true, true, 4, 2>, int8_tile_kernel<true, true, true, 6, 1>};
  static std::atomic<uint64_t> allowed[32];
  const int which = (l.P - 1) * 16 + (l.S > 1) * 8 + gated * 4 + (l.blocks == 1 ? 0 : l.blocks == 2 ? 1 : l.blocks == 4 ? 2 : 3);
  e = allow_shared(kernels[which], allowed[which], smem_optin);
  if (e != cudaSuccess) return e;
  if (l.blocks >= 4) {
    static std::atomic<int> regs[32];
    int n = regs[which].load(std::memory_order_relaxed);
    if (!n) {
      cudaFuncAttributes attr;
      e = cudaFuncGetAttributes(&attr, kernels[which]);
      if (e != cudaSuccess) return e;
      regs[which].store(n = attr.numRegs, std::memory_order_relaxed);
    }
    if (!int8_registers_fit(n)) return cudaErrorInvalidConfiguration;
  }
  const int fit = sms / l.P;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(l.P * (l.S > 1 ? l.T * l.S : l.T < fit ? l.T : fit));
  cfg.blockDim = dim3(kI8Threads);
  cfg.dynamicSmemBytes = 1024 + (size_t)l.stages * int8_stage_bytes(l) + sizeof(TileBars) + int8_extra_bytes(gated);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = l.P * l.S;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = l.P * l.S > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernels[which], mw, mw2, mx, p);
}

}  // namespace sesg
