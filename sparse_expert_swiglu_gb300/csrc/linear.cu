// y = act(x w^T + bias) [* (x w_mul^T + bias_mul)] [+ residual] on 16-bit x and w, fp32 sums.
//
// The features lie on the 128 TMEM lanes, the tokens on the columns: a tile is up to 256 features
// (two products of 128 lanes that share the token operand; with w_mul one of each matrix) by up to
// 256 tokens.  With few tokens the call is a stream of w, bound by HBM; with many it is bound by the
// tensor cores.  Where there are fewer tiles than SMs, a cluster of 2, 4 or 8 CTAs shares a tile
// along k: each CTA pushes its partial sums into the shared memory of the CTA that owns their features,
// which adds them in the order of k and runs the epilogue for them (no workspace, no
// count in global memory).  linear_plan chooses the tile and the cluster.
#include "activate.cuh"
#include "dense.cuh"
#include "dense_params.cuh"
#include "linear_plan.h"

namespace sesg {

namespace {

struct LinearArgs {
  int M, N, gated, bf16, kn, act, out_f32;
  int MT, NT, T;    // token tiles, tokens of a tile, tiles
  int rows;         // features of one product, <= 128
  int both;         // two products (always with w_mul)
  int wide;         // chunks of 64 k in a stage, one behind the other
  int KC, S;        // stages of a tile, CTAs (or CTA pairs) that share it along k
  int split;        // y as two 16-bit rows for each token, 2 t and 2 t + 1: the rounded value and the rest
  int pairs;        // x has two such rows for each token of y
  int groups;       // accumulators of a product: stage c of a round goes to c % groups
  int per;          // stages of a round (with KEEP)
  const void *bias, *bias_mul, *residual;
  void* y;
  DenseHead* head;
  int stages, acc_bufs, buf_cols, tmem_cols, stream;
  int own_x;        // the cluster's partial sums have memory of their own, behind the stages
  uint32_t tries;   // rounds of a wait
  int missing;      // diagnostics: the first CTA's stages wait for an arrival that does not come
};

// Tile t's feature and token tile.  Tiles that run together share operands: eight token tiles at a time go
// through all features, so that a wave of them is about as many features as tokens.
__device__ __forceinline__ void tile_at(int t, int T, int MT, int& ft, int& mt) {
  const int block = T / MT * kTogether, b = t / block, r = t - b * block;
  const int here = MT - b * kTogether < kTogether ? MT - b * kTogether : kTogether;
  ft = r / here;
  mt = b * kTogether + r - ft * here;
}

// The residual of W tokens of one feature; token i at offset at + i * N.
template <int W>
__device__ __forceinline__ void linear_residual(const LinearArgs& p, size_t at, int n, unsigned short (&r)[W]) {
  const unsigned short* from = reinterpret_cast<const unsigned short*>(p.residual) + at;
#pragma unroll
  for (int i = 0; i < W; ++i) r[i] = i < n ? from[(size_t)i * p.N] : (unsigned short)0;
}

// Residual and store of W tokens' values of one feature; token i at offset at + i * N.
template <int W, bool FULL>
__device__ __forceinline__ void linear_write(const LinearArgs& p, size_t at, int n, float (&v)[W],
                                             const unsigned short (&r)[W]) {
  if (p.residual) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] += from16(r[i], p.bf16);
  }
  if (p.out_f32) {
    float* y = reinterpret_cast<float*>(p.y) + at;
#pragma unroll
    for (int i = 0; i < W; ++i)
      if (FULL || i < n) y[(size_t)i * p.N] = v[i];
  } else {
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
}

// Epilogue of W tokens of one feature: v, and with w_mul m, are the sums, r the residual; n tokens from t0 exist.
template <int W>
__device__ __forceinline__ void linear_store(const LinearArgs& p, int feat, int t0, int n, float bias, float bias_mul,
                                             float (&v)[W], const float (&m)[W], const unsigned short (&r)[W]) {
#pragma unroll
  for (int i = 0; i < W; ++i) v[i] += bias;
  activate(v, p.act);
  if (p.gated) {
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] *= m[i] + bias_mul;
  }
  if (p.split) {
    unsigned short* y = reinterpret_cast<unsigned short*>(p.y) + (size_t)t0 * 2 * p.N + feat;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const unsigned short hi = to16(v[i], p.bf16);
      const float h = from16(hi, p.bf16);
      if (i < n) {
        y[(size_t)2 * i * p.N] = hi;
        y[(size_t)(2 * i + 1) * p.N] = isfinite(h) ? to16(v[i] - h, p.bf16) : (unsigned short)0;
      }
    }
    return;
  }
  const size_t at = (size_t)t0 * p.N + feat;
  if (n >= W) linear_write<W, true>(p, at, n, v, r);
  else linear_write<W, false>(p, at, n, v, r);
}

// The same where x has two rows for each token: their sums are added first.  (Without bias, act and w_mul.)
template <int W>
__device__ __forceinline__ void linear_store_pairs(const LinearArgs& p, int feat, int t0, int n, const float (&v)[W]) {
  float s[W / 2];
#pragma unroll
  for (int i = 0; i < W / 2; ++i) s[i] = v[2 * i] + v[2 * i + 1];
  const size_t at = (size_t)(t0 / 2) * p.N + feat;
  unsigned short r[W / 2];
  if (p.residual) linear_residual(p, at, n / 2, r);
  linear_write<W / 2, false>(p, at, n / 2, s, r);
}

// W columns of a product, its accumulators added.
template <int W>
__device__ __forceinline__ void linear_sums(uint32_t addr, int groups, int stride, float (&v)[W]) {
  tmem_ld(addr, v);
  tmem_wait(v);
  for (int g = 1; g < groups; ++g) {
    float t[W];
    tmem_ld(addr + g * stride, t);
    tmem_wait(t);
#pragma unroll
    for (int i = 0; i < W; ++i) v[i] += t[i];
  }
}

constexpr uint32_t kNoBlock = 0xffffffffu;

// A round's sums of this warp's blocks of 16 columns (at(b): the address of block b, kNoBlock: there is none), added to
// those of the rounds before; the last round's go back to where they were.  N columns at a time: as many as leave the
// kernel without a stack frame, with which a call takes 3.5 us longer.
template <int N, typename At>
__device__ __forceinline__ void linear_round(float (&acc)[8][16], bool last, At at) {
#pragma unroll
  for (int b = 0; b < 8; ++b) {
    const uint32_t a = at(b);
    if (a == kNoBlock) continue;  // the same for the whole warp
#pragma unroll
    for (int h = 0; h < 16; h += N) {
      float v[N];
      tmem_ld(a + h, v);
      tmem_wait(v);
#pragma unroll
      for (int i = 0; i < N; ++i) acc[b][h + i] += v[i];
    }
    if (last) tmem_st(a, acc[b]);
  }
}

// FEW: up to kFewTokens tokens and one tile for each CTA, whose epilogue takes 4 tokens at a time: a call this short
// pays for every line of code it fetches.  PAIR: CTA pairs (cta_group::2).  A tile then has up to 256 lanes for each product, 128 in each
// CTA, and either CTA fetches and keeps half of its tokens: with 100 to 500 tokens, where the bytes that
// an SM can take from L2 bound the products (300 tokens of 14336 gated features of K = 4096: 72 us, 78 without).
// SHARED: clusters share a tile along k; the one epilogue is not fetched with the other (an expert on 100 tokens, 2048 x
// 1408: 20.8 us against 21.9).
// KEEP: a tile's stages in rounds (LinearSums), whose sums this warp's threads add up; never with FEW.
template <bool FEW, bool PAIR, bool SHARED, bool KEEP>
__global__ void __launch_bounds__(kDnThreads, 1)
linear_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mw2,
              const __grid_constant__ CUtensorMap mx, const LinearArgs p) {
  extern __shared__ uint8_t raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  const int bytes_a = p.both ? kDnBytesA : kDnBytesA / 2;  // of a chunk; rows behind p.rows stay unwritten
  constexpr int P = PAIR ? 2 : 1;  // CTAs that run one product
  const uint32_t chunk_bytes = bytes_a + p.NT / P * 128, stage_bytes = p.wide * chunk_bytes;
  const int most = p.M < p.NT ? p.M : p.NT;  // tokens of a tile that exist
  const int load_rows = p.kn || p.N > p.rows ? p.rows : p.N;  // boxes are no higher than the operands
  const int load_toks = p.M < p.NT / P ? p.M : p.NT / P;
  const uint32_t load_bytes = P * p.wide * ((p.both ? 2 : 1) * load_rows + load_toks) * 128;
  // partial sums that a cluster's CTAs push here: behind the stages, or in them once they are free
  const int g4 = (most + 3) / 4, mats = p.gated ? 2 : 1;
  uint8_t* xsums = p.own_x ? ring + (size_t)p.stages * stage_bytes : ring;
  DenseBars* bars = reinterpret_cast<DenseBars*>(ring + (size_t)p.stages * stage_bytes +
                                                 (p.own_x ? (size_t)mats * g4 * 4096 : 0));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int S = SHARED ? p.S : 1, ns = p.stages, NT = p.NT;
  const int crank = PAIR || S > 1 ? (int)cluster_rank() : 0, half_of = PAIR ? crank & 1 : 0, lead = crank - half_of;
  const int rank = SHARED ? crank / P : 0;                                 // share of k
  const int first = blockIdx.x / (P * S), step = gridDim.x / (P * S);  // tiles of this CTA; S > 1: one
  const int kc0 = p.KC * rank / S, kc1 = p.KC * (rank + 1) / S;
  const int width = p.gated || !p.both ? p.rows : 2 * p.rows;  // features of a CTA in a tile
  int* status = &p.head->ctrl.status;
  const uint32_t ring_at = smem_addr(ring);

  if (tid == 0) {
    dn_init_bars(bars, p.tries, P * kDnEpi / 32, 1 + (p.missing && blockIdx.x == 0));
    mbar_init(&bars->xready, S);
    mbar_init(&bars->xfull, FEW ? 1 : 8);
    fence_barrier_init();
    tma_prefetch_map(&mw);
    tma_prefetch_map(&mx);
    if (p.gated) tma_prefetch_map(&mw2);
  }
  if (warp == 2) {
    if (PAIR) tmem_alloc_pair(&bars->tmem, p.tmem_cols);
    else tmem_alloc(&bars->tmem, p.tmem_cols);
  }
  tc_before_sync();
  __syncthreads();
  if (PAIR || S > 1) cluster_sync_all();  // the barriers are there before any CTA of the cluster uses them
  tc_after_sync();
  const uint32_t tmem = bars->tmem;
  // Before the wait: the next call's CTAs start while the last one's may still run (0.8 to 1.4 us of a short call behind
  // another).  This library's kernels touch no global memory before their own wait, but for the decode gather kernel's x,
  // which is complete when the kernel in front of it passes its wait.
  griddep_launch_dependents();
  griddep_wait();

  if (warp == 0) {
    if (elect_one()) {
      // w is read once when one tile of tokens covers them all
      const uint64_t pw = p.stream ? policy_evict_first() : policy_evict_normal();
      const uint64_t px = policy_evict_normal();
      const uint32_t full_at = PAIR ? peer_addr(smem_addr(&bars->full[0]), lead) : 0;
      int st = 0, issued = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = first; ok && t < p.T; t += step) {
        int ft, mt;
        tile_at(t, p.T, p.MT, ft, mt);
        const int f0 = (ft * P + half_of) * width, m0 = mt * NT + half_of * (NT / P);
        const CUtensorMap* m2 = p.gated ? &mw2 : &mw;
        const int f1 = p.gated ? f0 : f0 + p.rows;
        for (int kc = kc0; kc < kc1; ++kc) {
          if (!dn_wait(&bars->empty[st], ph ^ 1, bars)) {
            dn_fail(bars, status);
            ok = false;
            break;
          }
          uint64_t* full = &bars->full[st];
          if (crank == lead) mbar_arrive_expect_tx(full, load_bytes);
          ++issued;
          // a pair's copies count on the first CTA's barrier
          auto copy = [&](uint32_t to, const CUtensorMap* m, int c0, int c1, uint64_t pol) {
            if constexpr (PAIR) tma_2d_pair(to, m, c0, c1, full_at + st * 8, pol);
            else tma_2d(to, m, c0, c1, full, pol);
          };
          uint32_t a = ring_at + st * stage_bytes;
          for (int c = 0; c < p.wide; ++c, a += chunk_bytes) {
            const int k = (kc * p.wide + c) * kDnChunk;
            if (!p.kn) {
              copy(a, &mw, k, f0, pw);
              if (p.both) copy(a + kDnBytesA / 2, m2, k, f1, pw);
            } else {
              for (int i = 0; i < p.rows; i += 64) {
                copy(a + i * 128, &mw, f0 + i, k, pw);
                if (p.both) copy(a + kDnBytesA / 2 + i * 128, m2, f1 + i, k, pw);
              }
            }
            copy(a + bytes_a, &mx, k, m0, px);
          }
          if (++st == ns) {
            st = 0;
            ph ^= 1;
          }
        }
      }
      // No copy of this CTA is in flight when it ends: the last stages have come.  A pair has used every copy, unless
      // it gave up: no barrier of this CTA counts them.
      if (PAIR && dn_aborted(bars)) dn_settle();
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
      const uint32_t desc = mma_desc(NT, p.bf16, p.kn, P * kDnHalf);
      auto commit = [&](uint64_t* bar) {
        if constexpr (PAIR) mma_commit_pair(bar, lead);
        else mma_commit(bar);
      };
      const int grp_cols = (p.both ? 2 : 1) * NT;
      int st = 0, buf = 0;
      uint32_t ph = 0, tph = 0;
      bool ok = true, open = false;
      for (int t = first; ok && t < p.T; t += step) {
        for (int kr = kc0, end; ok && kr < kc1; kr = end) {
          end = KEEP && kr + p.per < kc1 ? kr + p.per : kc1;
          if (!(PAIR ? cluster_wait(&bars->tempty[buf], tph ^ 1, bars) : dn_wait(&bars->tempty[buf], tph ^ 1, bars))) {
            dn_fail(bars, status);
            ok = false;
            break;
          }
          tc_after_sync();
          int grp = 0;
          for (int kc = kr; kc < end; ++kc) {
            if (!dn_wait(&bars->full[st], ph, bars)) {
              dn_fail(bars, status);
              ok = false;
              break;
            }
            tc_after_sync();
            const uint32_t a = ring_at + st * stage_bytes;
            const uint32_t d0 = tmem + buf * p.buf_cols + grp * grp_cols;
            for (int c = 0; c < p.wide; ++c)
              dn_stage_products<PAIR>(a + c * chunk_bytes, a + c * chunk_bytes + bytes_a, d0, d0 + NT, desc, p.kn,
                                      c == 0 && kc - kr < (KEEP ? 1 : p.groups), p.both);
            commit(&bars->empty[st]);
            open = true;
            if (!KEEP && ++grp == p.groups) grp = 0;
            if (++st == ns) {
              st = 0;
              ph ^= 1;
            }
          }
          if (!ok) break;
          commit(&bars->tfull[buf]);
          if (++buf == p.acc_bufs) {
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
  } else if (warp >= 4) {
    // Lanes 32 (warp % 4) ... are this warp's.  Of the two warps that have them, each takes one of the
    // two products, or, where both products belong to one feature (or there is one), every other 16 tokens.
    constexpr int W = FEW || (KEEP && !SHARED) ? 4 : 16;  // tokens at a time
    const int q = warp & 3, half = (warp - 4) >> 2, etid = tid - 128;
    const bool by_tok = p.gated || !p.both;
    const int tok0 = by_tok ? 16 * half : 0, tok_step = by_tok ? 32 : 16;
    const int row = q * 32 + lane;
    const int grp_cols = (p.both ? 2 : 1) * NT;
    const int groups = KEEP ? 1 : kc1 - kc0 < p.groups ? kc1 - kc0 : p.groups;
    const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + (by_tok ? 0 : half * NT);
    int buf = 0;
    uint32_t tph = 0;
    for (int t = first; t < p.T; t += step) {
      // this warp's columns of the sets of accumulators that have been read
      auto release = [&] {
        tc_before_sync();
        __syncwarp();
        if (lane == 0) {
          if (PAIR) peer_arrive(peer_addr(smem_addr(&bars->tempty[buf]), lead));
          else mbar_arrive(&bars->tempty[buf]);
        }
        if (++buf == p.acc_bufs) {
          buf = 0;
          tph ^= 1;
        }
      };
      if constexpr (KEEP) {
        float acc[8][16];
#pragma unroll
        for (int b = 0; b < 8; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[b][i] = 0.f;
        bool ok = true;
        for (int kr = kc0; kr < kc1; kr += p.per) {
          ok = dn_wait(&bars->tfull[buf], tph, bars);
          if (!ok) dn_fail(bars, status);
          ok = !dn_any(1, kDnEpi, !ok);  // one decision for the warps
          if (!ok) break;
          tc_after_sync();
          const bool last = kr + p.per >= kc1;
          linear_round<SHARED ? 16 : 8>(acc, last, [&](int b) {
            const int n0 = tok0 + tok_step * (p.gated ? b & 3 : b);
            return n0 < NT ? lanes + buf * p.buf_cols + (p.gated ? b >> 2 : 0) * NT + n0 : kNoBlock;
          });
          if (last) tmem_stored();
          else release();
        }
        if (!ok) break;
      }
      int ft, mt;
      tile_at(t, p.T, p.MT, ft, mt);
      const int m0 = mt * NT;
      const int nt = p.M - m0 < NT ? p.M - m0 : NT;  // tokens of this tile
      if constexpr (!SHARED) {
        const int feat = (ft * P + half_of) * width + (by_tok ? 0 : half * p.rows) + row;
        const bool on = row < p.rows && feat < p.N;
        const float ba = p.bias && on ? ld16(p.bias, feat, p.bf16) : 0.f;
        const float bb = p.bias_mul && on ? ld16(p.bias_mul, feat, p.bf16) : 0.f;
        // the residual is asked for ahead, one step before it is added
        const bool with_r = p.residual && on && !p.pairs;
        unsigned short r[W], rn[W];
        if (with_r && tok0 < nt) linear_residual(p, (size_t)(m0 + tok0) * p.N + feat, nt - tok0, rn);
        if constexpr (!KEEP) {
          const bool ok = dn_wait(&bars->tfull[buf], tph, bars);
          if (!ok) dn_fail(bars, status);
          if (dn_any(1, kDnEpi, !ok)) break;  // one decision for the warps
          tc_after_sync();
        }
        const uint32_t d0 = lanes + buf * p.buf_cols;
        for (int n0 = tok0; n0 < nt; n0 += tok_step) {
#pragma unroll 1
          for (int i = n0; i < nt && i < n0 + 16; i += W) {
            float v[W], m[W];
            const int next = i + W < n0 + 16 ? i + W : n0 + tok_step;
#pragma unroll
            for (int j = 0; j < W; ++j) r[j] = rn[j];
            if (with_r && next < nt) linear_residual(p, (size_t)(m0 + next) * p.N + feat, nt - next, rn);
            linear_sums(d0 + i, groups, grp_cols, v);
            if (p.gated) linear_sums(d0 + NT + i, groups, grp_cols, m);
            if (on && p.pairs) linear_store_pairs(p, feat, m0 + i, nt - i, v);
            else if (on) linear_store(p, feat, m0 + i, nt - i, ba, bb, v, m, r);
            __syncwarp();
          }
        }
        release();
      } else {
        // The warp pair's unit 2 q + half of sums belongs to the share unit * S / 8's CTA with the same lanes: 4 tokens of a
        // feature are 16 bytes at [unit of the owner][rank][matrix][4 tokens][lane], with room for all tokens in a unit.
        // Few tokens' stores count their bytes on the owner's barrier themselves (one token of 4096 x 4096 9.35 us
        // against 9.50); many go faster as plain stores with one arrival for each warp (300 tokens of 14336 down rows 39.8
        // against 41.3).
        const uint32_t unit_bytes = mats * g4 * 512;
        const int per = 8 / S, unit = 2 * q + half;
        auto groups4 = [&](int h) {  // groups of 4 tokens that exist in a unit of half h
          if (!by_tok) return (nt + 3) / 4;
          int n = 0;
          for (int n0 = 16 * h; n0 < nt; n0 += 32) n += ((nt - n0 < 16 ? nt - n0 : 16) + 3) / 4;
          return n;
        };
        bool ok = KEEP || dn_wait(&bars->tfull[0], 0, bars);
        if (etid == 0 && ok) {
          if (FEW) {
            uint32_t bytes = 0;
            for (int i = 0; i < per; ++i) bytes += S * mats * groups4((rank * per + i) & 1) * 512;
            mbar_arrive_expect_tx(&bars->xfull, bytes);
          }
          if (!p.own_x)
            for (int i = 0; i < S; ++i) peer_arrive(peer_addr(smem_addr(&bars->xready), P * i + half_of));
        }
        if (!p.own_x) ok = ok && cluster_wait(&bars->xready, 0, bars);
        if (!ok) dn_fail(bars, status);
        if (dn_any(1, kDnEpi, !ok)) break;
        tc_after_sync();
        {
          const int owner = unit / per;
          const uint32_t d0 = lanes + (KEEP ? buf * p.buf_cols : 0);
          const int peer = P * owner + half_of;
          uint32_t to = peer_addr(smem_addr(xsums), peer) + ((unit - owner * per) * S + rank) * unit_bytes + lane * 16;
          const uint32_t bar = peer_addr(smem_addr(&bars->xfull), peer);
          for (int n0 = tok0; n0 < nt; n0 += tok_step) {
#pragma unroll 1
            for (int i = n0; i < nt && i < n0 + 16; i += W) {
#pragma unroll 1
              for (int mat = 0; mat < mats; ++mat) {
                float v[W];
                linear_sums(d0 + mat * NT + i, groups, grp_cols, v);
#pragma unroll
                for (int j = 0; j < W; j += 4)
                  if (i + j < nt) {
                    if (FEW) peer_store(to + (mat * g4 + j / 4) * 512, v + j, bar);
                    else peer_store(to + (mat * g4 + j / 4) * 512, v + j);
                  }
              }
              to += W / 4 * 512;
            }
          }
          __syncwarp();
          if (!FEW && lane == 0) peer_arrive(bar);  // releases the warp's stores
        }
        ok = cluster_wait(&bars->xfull, 0, bars);
        if (!ok) dn_fail(bars, status);
        if (dn_any(1, kDnEpi, !ok)) break;
        {
          // S warps for each of this CTA's units, taking its groups of 4 tokens in turn
          const int w = warp - 4, ul = w / S, u = rank * per + ul, uq = u >> 1, uh = u & 1;
          const int feat = (ft * P + half_of) * width + (by_tok ? 0 : uh * p.rows) + uq * 32 + lane;
          const bool on = uq * 32 + lane < p.rows && feat < p.N;
          const float ba = p.bias && on ? ld16(p.bias, feat, p.bf16) : 0.f;
          const float bb = p.bias_mul && on ? ld16(p.bias_mul, feat, p.bf16) : 0.f;
          const int n4 = groups4(uh);
          const uint8_t* from = xsums + (size_t)ul * S * unit_bytes + lane * 16;
          for (int i = w % S; i < n4; i += S) {
            const int n0 = by_tok ? 16 * uh + 32 * (i >> 2) + 4 * (i & 3) : 4 * i;
            unsigned short r[4];
            if (p.residual && on && !p.pairs) linear_residual(p, (size_t)(m0 + n0) * p.N + feat, nt - n0, r);
            float v[4] = {0.f, 0.f, 0.f, 0.f}, m[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
            for (int s = 0; s < S; ++s) {
              const float4 a = *reinterpret_cast<const float4*>(from + s * unit_bytes + i * 512);
              v[0] += a.x;
              v[1] += a.y;
              v[2] += a.z;
              v[3] += a.w;
              if (p.gated) {
                const float4 b = *reinterpret_cast<const float4*>(from + s * unit_bytes + (g4 + i) * 512);
                m[0] += b.x;
                m[1] += b.y;
                m[2] += b.z;
                m[3] += b.w;
              }
            }
            if (on && p.pairs) linear_store_pairs(p, feat, m0 + n0, nt - n0, v);
            else if (on) linear_store(p, feat, m0 + n0, nt - n0, ba, bb, v, m, r);
          }
        }
      }
    }
  }
  __syncwarp();
  tc_before_sync();
  __syncthreads();
  if (PAIR || S > 1) {
    cluster_sync_all();  // no CTA leaves while another may store into it
    if (dn_aborted(bars)) dn_settle();  // stores that this CTA did not wait for
  }
  tc_after_sync();
  if (warp == 2) {
    if (PAIR) tmem_free_pair(tmem, p.tmem_cols);
    else tmem_free(tmem, p.tmem_cols);
  }
}

// ---------------------------------------------------------------------------
// Many tokens: CTA pairs (cta_group::2).  Here the tokens lie on the lanes, 128 of a tile's 256 in each
// CTA, and up to 256 columns of weights are the other operand, half from each CTA's shared memory (with
// w_mul: rows of w from the first CTA, the same rows of w_mul from the second, so that one thread has both
// sums of a feature).  A stage is up to 32 KB for 4 products of up to 128 clocks, half of what one CTA alone would
// have to fetch and read, and the columns of sums are doubled: the epilogue of a tile runs under the next one's
// products, and stores 16 bytes of a token's row at a time.  The number of columns is chosen so that the
// tiles fill whole waves.
// ---------------------------------------------------------------------------
constexpr int kPairStage = 2 * kDnHalf * kDnChunk * 2;
constexpr int kPairStages = 7;

struct PairArgs {
  int M, N, gated, bf16, kn, act, out_f32;
  int MT, T, KC;
  int rows;         // of weights from each CTA: a multiple of 16 (with w_mul 32), <= 128
  int per;          // chunks of a round (with KEEP)
  int sectors;      // every 16 features of a token's row start on a 32-byte boundary of y
  const void *bias, *bias_mul, *residual;
  void* y;
  DenseHead* head;
  uint32_t tries;   // as in LinearArgs
  int missing;
};

// 8 neighbouring features of a token from a 16-bit array, added or assigned; n of them exist.
__device__ __forceinline__ void load8(const void* base, size_t at, int n, int bf16, float (&v)[8]) {
  uint4 t = make_uint4(0, 0, 0, 0);
  if (n > 0) t = *reinterpret_cast<const uint4*>(reinterpret_cast<const unsigned short*>(base) + at);
  const uint32_t w[4] = {t.x, t.y, t.z, t.w};
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = from16((unsigned short)(w[i / 2] >> (16 * (i & 1))), bf16);
}

// 32 bytes at a time: whole sectors (32-byte aligned)
__device__ __forceinline__ void store32(void* to, const uint32_t (&w)[8]) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(to), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

// Epilogue of 16 neighbouring features of one token (N a multiple of 8: of each 8 all exist or none).
__device__ __forceinline__ void pair_store(const PairArgs& p, size_t row, int feat, float (&v)[16], const float (&m)[16],
                                           const uint4 (&r)[2]) {
  float t[8];
  if (p.bias) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      load8(p.bias, feat + 8 * h, p.N - feat - 8 * h, p.bf16, t);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[8 * h + i] += t[i];
    }
  }
  activate(v, p.act);
  if (p.gated) {
    if (p.bias_mul) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        load8(p.bias_mul, feat + 8 * h, p.N - feat - 8 * h, p.bf16, t);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[8 * h + i] *= m[8 * h + i] + t[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] *= m[i];
    }
  }
  const size_t at = row * p.N + feat;
  if (p.residual) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t w[4] = {r[h].x, r[h].y, r[h].z, r[h].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) v[8 * h + i] += from16((unsigned short)(w[i / 2] >> (16 * (i & 1))), p.bf16);
    }
  }
  if (p.sectors) {
    uint32_t w[8];
    if (p.out_f32) {
      float* y = reinterpret_cast<float*>(p.y) + at;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = __float_as_uint(v[8 * h + i]);
        store32(y + 8 * h, w);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        w[i] = (uint32_t)to16(v[2 * i], p.bf16) | (uint32_t)to16(v[2 * i + 1], p.bf16) << 16;
      store32(reinterpret_cast<unsigned short*>(p.y) + at, w);
    }
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (feat + 8 * h >= p.N) break;
    if (p.out_f32) {
      float4* y = reinterpret_cast<float4*>(reinterpret_cast<float*>(p.y) + at + 8 * h);
      y[0] = make_float4(v[8 * h], v[8 * h + 1], v[8 * h + 2], v[8 * h + 3]);
      y[1] = make_float4(v[8 * h + 4], v[8 * h + 5], v[8 * h + 6], v[8 * h + 7]);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = (uint32_t)to16(v[8 * h + 2 * i], p.bf16) | (uint32_t)to16(v[8 * h + 2 * i + 1], p.bf16) << 16;
      *reinterpret_cast<uint4*>(reinterpret_cast<unsigned short*>(p.y) + at + 8 * h) = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// KEEP: a tile's chunks in rounds (LinearSums), whose sums this warp's threads add up.
template <bool KEEP>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kDnThreads, 1)
linear_pair_kernel(const __grid_constant__ CUtensorMap mw, const __grid_constant__ CUtensorMap mw2,
                   const __grid_constant__ CUtensorMap mx, const PairArgs p) {
  extern __shared__ uint8_t raw[];
  // the same offset in both CTAs: the products address both CTAs' stages by it
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
  DenseBars* bars = reinterpret_cast<DenseBars*>(ring + (size_t)kPairStages * kPairStage);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_rank(), first = blockIdx.x / 2, step = gridDim.x / 2;
  const int width = p.gated ? p.rows : 2 * p.rows;  // features of a tile
  const int load_rows = p.kn ? (p.rows + 63) / 64 * 64 : p.rows;
  int* status = &p.head->ctrl.status;
  const uint32_t ring_at = smem_addr(ring);

  if (tid == 0) {
    dn_init_bars(bars, p.tries, 2 * kDnEpi / 32, 1 + (p.missing && blockIdx.x == 0));
    tma_prefetch_map(&mw);
    tma_prefetch_map(&mx);
    if (p.gated) tma_prefetch_map(&mw2);
  }
  if (warp == 2) tmem_alloc_pair(&bars->tmem, 512);
  tc_before_sync();
  __syncthreads();
  cluster_sync_all();
  tc_after_sync();
  const uint32_t tmem = bars->tmem;
  griddep_wait();
  griddep_launch_dependents();

  if (warp == 0) {
    if (elect_one()) {
      const uint64_t pol = policy_evict_normal();
      const CUtensorMap* mb = p.gated && rank ? &mw2 : &mw;
      const uint32_t full_at = peer_addr(smem_addr(&bars->full[0]), 0);
      int st = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (int t = first; ok && t < p.T; t += step) {
        int ft, mt;
        tile_at(t, p.T, p.MT, ft, mt);
        const int m0 = mt * 2 * kDnHalf + rank * kDnHalf, f0 = ft * width + (p.gated ? 0 : rank * p.rows);
        for (int kc = 0; kc < p.KC; ++kc) {
          if (!dn_wait(&bars->empty[st], ph ^ 1, bars)) {
            dn_fail(bars, status);
            ok = false;
            break;
          }
          if (rank == 0) mbar_arrive_expect_tx(&bars->full[st], 2 * (kPairStage / 2 + load_rows * 128));
          const uint32_t full = full_at + st * 8;
          const uint32_t a = ring_at + st * kPairStage, b = a + kPairStage / 2;
          const int k = kc * kDnChunk;
          tma_2d_pair(a, &mx, k, m0, full, pol);
          if (!p.kn) {
            tma_2d_pair(b, mb, k, f0, full, pol);
          } else {
            for (int i = 0; i < load_rows; i += 64) tma_2d_pair(b + i * 128, mb, f0 + i, k, full, pol);
          }
          if (++st == kPairStages) {
            st = 0;
            ph ^= 1;
          }
        }
      }
      // After an abort copies may be in flight that no barrier of this CTA counts.  (Without one, every copy has been used.)
      if (dn_aborted(bars)) dn_settle();
    }
  } else if (warp == 1) {
    if (rank == 0 && elect_one()) {
      // 256 lanes (both CTAs) by 2 rows columns
      const uint32_t desc = (1u << 4) | ((uint32_t)p.bf16 << 7) | ((uint32_t)p.bf16 << 10) | ((uint32_t)p.kn << 16) |
                            ((uint32_t)(2 * p.rows >> 3) << 17) | ((256u >> 4) << 24);
      int st = 0, buf = 0;
      uint32_t ph = 0, tph = 0;
      bool ok = true, open = false;
      for (int t = first; ok && t < p.T; t += step) {
        for (int kr = 0, end; ok && kr < p.KC; kr = end) {
          end = KEEP && kr + p.per < p.KC ? kr + p.per : p.KC;
          if (!cluster_wait(&bars->tempty[buf], tph ^ 1, bars)) {
            dn_fail(bars, status);
            ok = false;
            break;
          }
          tc_after_sync();
          const uint32_t d = tmem + buf * 256;
          for (int kc = kr; kc < end; ++kc) {
            if (!dn_wait(&bars->full[st], ph, bars)) {
              dn_fail(bars, status);
              ok = false;
              break;
            }
            tc_after_sync();
            const uint32_t a = ring_at + st * kPairStage;
            const uint64_t ad = smem_desc(a, 16), bd = smem_desc(a + kPairStage / 2, p.kn ? 8192 : 16);
            const uint32_t step = p.kn ? 128 : 2;
#pragma unroll
            for (int ks = 0; ks < kDnChunk / 16; ++ks)
              mma_f16_pair(d, ad + ks * 2, bd + ks * step, desc, kc > kr || ks > 0);
            mma_commit_pair(&bars->empty[st]);
            open = true;
            if (++st == kPairStages) {
              st = 0;
              ph ^= 1;
            }
          }
          if (!ok) break;
          mma_commit_pair(&bars->tfull[buf]);
          buf ^= 1;
          tph ^= buf == 0;
        }
      }
      if (open) {  // every product is done before TMEM is given back
        mma_commit_pair(&bars->drain);
        dn_drain(&bars->drain, 0, kWaitTries);
      }
    }
  } else if (warp >= 4) {
    const int q = warp & 3, half = (warp - 4) >> 2;
    const int cols = p.gated ? p.rows / 2 : p.rows;  // features of this warp
    int buf = 0;
    uint32_t tph = 0;
    for (int t = first; t < p.T; t += step) {
      const uint32_t lanes = tmem + ((uint32_t)(q * 32) << 16) + half * cols;
      auto release = [&] {
        tc_before_sync();
        __syncwarp();
        if (lane == 0) peer_arrive(peer_addr(smem_addr(&bars->tempty[buf]), 0));
        buf ^= 1;
        tph ^= buf == 0;
      };
      if constexpr (KEEP) {
        float acc[8][16];
#pragma unroll
        for (int b = 0; b < 8; ++b)
#pragma unroll
          for (int i = 0; i < 16; ++i) acc[b][i] = 0.f;
        bool ok = true;
        for (int kr = 0; kr < p.KC; kr += p.per) {
          ok = dn_wait(&bars->tfull[buf], tph, bars);
          if (!ok) dn_fail(bars, status);
          ok = !dn_any(1, kDnEpi, !ok);  // one decision for the warps
          if (!ok) break;
          tc_after_sync();
          const bool last = kr + p.per >= p.KC;
          linear_round<4>(acc, last, [&](int b) {
            const int c = 16 * (p.gated ? b & 3 : b);
            return c < cols ? lanes + buf * 256 + (p.gated ? b >> 2 : 0) * p.rows + c : kNoBlock;
          });
          if (last) tmem_stored();
          else release();
        }
        if (!ok) break;
      }
      int ft, mt;
      tile_at(t, p.T, p.MT, ft, mt);
      const int tok = mt * 2 * kDnHalf + rank * kDnHalf + q * 32 + lane;
      const int f0 = ft * width + half * cols;
      // the residual is asked for ahead, one step before it is added
      uint4 r[2], rn[2];
      auto residual = [&](int c) {
        if (!p.residual || tok >= p.M) return;
        const unsigned short* from = reinterpret_cast<const unsigned short*>(p.residual) + (size_t)tok * p.N + f0 + c;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (f0 + c + 8 * h < p.N) rn[h] = *reinterpret_cast<const uint4*>(from + 8 * h);
      };
      residual(0);
      if constexpr (!KEEP) {
        const bool ok = dn_wait(&bars->tfull[buf], tph, bars);
        if (!ok) dn_fail(bars, status);
        if (dn_any(1, kDnEpi, !ok)) break;
        tc_after_sync();
      }
      const uint32_t d = lanes + buf * 256;
      for (int c = 0; c < cols && f0 + c < p.N; c += 16) {
        float v[16], m[16];
        r[0] = rn[0];
        r[1] = rn[1];
        if (c + 16 < cols) residual(c + 16);
        tmem_ld(d + c, v);
        if (p.gated) tmem_ld(d + p.rows + c, m);
        tmem_wait(v);
        if (p.gated) tmem_wait(m);
        if (tok < p.M) pair_store(p, tok, f0 + c, v, m, r);
        __syncwarp();
      }
      release();
    }
  }
  __syncwarp();
  tc_before_sync();
  __syncthreads();
  cluster_sync_all();  // no CTA leaves while the other's copies or arrivals may reach it
  if (dn_aborted(bars)) dn_settle();
  tc_after_sync();
  if (warp == 2) tmem_free_pair(tmem, 512);
}

constexpr size_t kHeadBytes = (sizeof(DenseHead) + 255) / 256 * 256;

}  // namespace

size_t linear_ws_bytes() { return kHeadBytes; }

static cudaError_t launch_linear_pair(const LinearCall& c, const LinearPlan& l, void* ws, int sms, int smem_optin,
                                      cudaStream_t st) {
  const bool gated = c.w_mul != nullptr;
  CUtensorMap mw, mw2, mx;
  const uint64_t cols = c.kn ? c.N : c.K, rows = c.kn ? c.K : c.N;
  const uint32_t box = c.kn ? kDnChunk : l.rows;
  cudaError_t e = dense_map(&mw, c.w, c.bf16, cols, rows, c.w_stride, 0, 0, box);
  if (e != cudaSuccess) return e;
  mw2 = mw;
  if (gated) e = dense_map(&mw2, c.w_mul, c.bf16, cols, rows, c.w_mul_stride, 0, 0, box);
  if (e == cudaSuccess) e = dense_map(&mx, c.x, c.bf16, c.K, c.M, c.K, 0, 0, kDnHalf);
  if (e != cudaSuccess) return e;
  PairArgs p;
  p.M = c.M;
  p.N = c.N;
  p.gated = gated;
  p.bf16 = c.bf16;
  p.kn = c.kn;
  p.act = c.act;
  p.out_f32 = c.out_f32;
  p.MT = l.MT;
  p.T = l.T;
  p.rows = l.rows;
  p.sectors = c.N % 16 == 0 && (uintptr_t)c.y % 32 == 0;  // y itself may start on 16 bytes
  p.KC = (c.K + kDnChunk - 1) / kDnChunk;
  p.bias = c.bias;
  p.bias_mul = c.bias_mul;
  p.residual = c.residual;
  p.y = c.y;
  p.head = reinterpret_cast<DenseHead*>(ws);
  p.tries = c.tries ? c.tries : kWaitTries;
  p.missing = c.tries > 0;
  const size_t smem = 1024 + (size_t)kPairStages * kPairStage + sizeof(DenseBars);
  p.per = sum_chunks(c.out_f32);
  const bool keep = p.KC > p.per;
  static std::atomic<uint64_t> allowed[2];
  const auto kernel = keep ? linear_pair_kernel<true> : linear_pair_kernel<false>;
  e = allow_shared(kernel, allowed[keep], smem_optin);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(2 * (p.T < sms / 2 ? p.T : sms / 2));
  cfg.blockDim = dim3(kDnThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, mw, mw2, mx, p);
}

cudaError_t launch_linear(const LinearCall& c, void* ws, int sms, int smem_optin, cudaStream_t st) {
  const bool gated = c.w_mul != nullptr;
  const int room = smem_optin - 1024 - (int)sizeof(DenseBars);
  const LinearPlan& l = linear_plan(c.M, c.N, c.K, gated, c.kn, !c.split && !c.pairs, c.out_f32, sms, room);
  if (!l.S) return cudaErrorInvalidValue;
  if (l.by_token) return launch_linear_pair(c, l, ws, sms, smem_optin, st);
  CUtensorMap mw, mw2, mx;
  const uint64_t cols = c.kn ? c.N : c.K, rows = c.kn ? c.K : c.N;
  // rows behind the last one would be slow to fetch where every tile has them (1542 x 18, K = 1400: 34 us
  // with boxes of 128 rows, 10 with 18)
  const uint32_t box = c.kn ? kDnChunk : c.N < l.rows ? c.N : l.rows;
  cudaError_t e = dense_map(&mw, c.w, c.bf16, cols, rows, c.w_stride, 0, 0, box);
  if (e != cudaSuccess) return e;
  mw2 = mw;
  if (gated) e = dense_map(&mw2, c.w_mul, c.bf16, cols, rows, c.w_mul_stride, 0, 0, box);
  if (e == cudaSuccess) e = dense_map(&mx, c.x, c.bf16, c.K, c.M, c.K, 0, 0, c.M < l.NT / l.P ? c.M : l.NT / l.P);
  if (e != cudaSuccess) return e;
  LinearArgs p;
  p.M = c.M;
  p.N = c.N;
  p.gated = gated;
  p.bf16 = c.bf16;
  p.kn = c.kn;
  p.act = c.act;
  p.out_f32 = c.out_f32;
  p.MT = l.MT;
  p.NT = l.NT;
  p.T = l.T;
  p.rows = l.rows;
  p.both = l.both;
  p.wide = l.wide;
  p.KC = ((c.K + kDnChunk - 1) / kDnChunk + l.wide - 1) / l.wide;
  p.S = l.S;
  p.split = c.split;
  p.pairs = c.pairs;
  p.bias = c.bias;
  p.bias_mul = c.bias_mul;
  p.residual = c.residual;
  p.y = c.y;
  p.head = reinterpret_cast<DenseHead*>(ws);
  p.tries = c.tries ? c.tries : kWaitTries;
  p.missing = c.tries > 0;
  const int stage = l.wide * ((l.both ? kDnBytesA : kDnBytesA / 2) + l.NT / l.P * 128);
  bool own_x;
  p.stages = linear_stages(l, c.M, gated, room, own_x);
  p.own_x = own_x;
  LinearSums sums;
  if (!linear_sums(l, c.K, c.out_f32, sums)) return cudaErrorInvalidValue;
  p.acc_bufs = sums.bufs;
  p.groups = sums.groups;
  p.per = sums.per;
  p.buf_cols = p.groups * (l.both ? 2 : 1) * l.NT;
  p.tmem_cols = 32;
  while (p.tmem_cols < sums.cols) p.tmem_cols *= 2;
  p.stream = l.MT == 1;
  const int ctas = l.P * (l.S > 1 ? l.T * l.S : l.T < sms / l.P ? l.T : sms / l.P);
  const size_t smem = 1024 + (size_t)p.stages * stage + sizeof(DenseBars) + (own_x ? linear_sum_bytes(l, c.M, gated) : 0);
  static std::atomic<uint64_t> allowed[10];
  const bool few = l.P == 1 && !sums.keep && l.NT <= kFewTokens && l.S * l.T <= sms;
  const int which = (few ? 8 : (l.P == 2 ? 4 : 0) + (sums.keep ? 2 : 0)) + (l.S > 1);
  constexpr decltype(&linear_kernel<false, false, false, false>) kernels[10] = {
      linear_kernel<false, false, false, false>, linear_kernel<false, false, true, false>,
      linear_kernel<false, false, false, true>,  linear_kernel<false, false, true, true>,
      linear_kernel<false, true, false, false>,  linear_kernel<false, true, true, false>,
      linear_kernel<false, true, false, true>,   linear_kernel<false, true, true, true>,
      linear_kernel<true, false, false, false>,  linear_kernel<true, false, true, false>};
  const auto kernel = kernels[which];
  e = allow_shared(kernel, allowed[which], smem_optin);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(kDnThreads);
  cfg.dynamicSmemBytes = smem;
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
  return cudaLaunchKernelEx(&cfg, kernel, mw, mw2, mx, p);
}

}  // namespace sesg
