// Shared parts of the kernels on uncompressed 16-bit weights (linear.cu, dense_layer.cu).
//
// The weights stream through tcgen05 as tiles: D[feature][token] += W[feature][k] x[token][k].  They
// are the 128-row operand A, so that one token costs no more than 16 (the smallest N); the tokens are
// operand B.  (Only the kernel for many tokens turns this round, linear.cu.)  One CTA per SM; a TMA warp
// fills a ring of stages of 64 k or a multiple of it (A: one or two tiles of up to 128 features; B: token rows
// of 128 bytes), one elected thread issues the products into TMEM, eight warps read the sums back.
// Every operand is stored with the 128-byte swizzle.
//
// Work that does not fill the SMs is cut along k: in linear.cu a cluster's CTAs share a tile and join
// their sums in shared memory; in the layer's one kernel the tiles behind the last full wave are cut into
// equal shares for all CTAs, joined in global memory (Sched).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>

#include "dense_plan.h"
#include "params.cuh"

namespace sesg {

// ---------------------------------------------------------------------------
// workspace head, the same for every call on uncompressed weights: Ctrl, the grid
// barriers' counts and the shares' counts, all zero between calls
// ---------------------------------------------------------------------------
struct DenseHead {
  Ctrl ctrl;
  unsigned bar[8];                 // grid barriers of the layer kernel
  unsigned tok[64];                // router slices done, per token
  unsigned pad[64 - 16];
  unsigned cnt[kDnMaxCtas];        // shares done, per split tile
};

struct Seg {
  int t, k0, k1;
};

struct SegIter {
  Sched s;
  int c, t, i0, i1;
  __device__ SegIter(const Sched& sc, int cta) : s(sc), c(cta), t(cta) {
    i0 = (int)((long long)cta * sc.q < sc.total ? cta * sc.q : sc.total);
    i1 = i0 + sc.q < sc.total ? i0 + sc.q : sc.total;
  }
  __device__ bool next(Seg& g) {
    if (t < s.dp) {
      g.t = t;
      g.k0 = 0;
      g.k1 = s.KC;
      t += s.P;
      return true;
    }
    if (i0 >= i1) return false;
    const int r = i0 / s.KC;
    g.t = s.dp + r;
    g.k0 = i0 - r * s.KC;
    g.k1 = g.k0 + i1 - i0 < s.KC ? g.k0 + i1 - i0 : s.KC;
    i0 += g.k1 - g.k0;
    return true;
  }
};

// ---------------------------------------------------------------------------
// tcgen05, TMA
// ---------------------------------------------------------------------------
// Shared-memory operand descriptor, 128-byte swizzle.  Rows along k (128 bytes per row):
// groups of 8 rows are 1024 bytes apart.  Rows along the other axis (the operand lies
// [k][64 features]): groups of 8 k are 1024 bytes apart, groups of 64 features `lead`.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lead) {
  return (uint64_t)((addr & 0x3FFFF) >> 4) | ((uint64_t)(lead >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
         (1ull << 46) | (2ull << 61);
}
// fp32 sums, both operands fp16 (bf16 = 0) or bf16, A's rows along k (a_mn = 0) or not
__device__ __forceinline__ uint32_t mma_desc(int n, int bf16, int a_mn, int lanes = kDnHalf) {
  return (1u << 4) | ((uint32_t)bf16 << 7) | ((uint32_t)bf16 << 10) | ((uint32_t)a_mn << 15) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(lanes >> 4) << 24);
}
__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(desc), "r"(add)
      : "memory");
}
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void tmem_alloc(uint32_t* at, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(at)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
__device__ __forceinline__ void tc_before_sync() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after_sync() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
// W columns of this warp's 32 lanes; the values are there after tmem_wait
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr));
#pragma unroll
  for (int i = 0; i < 16; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&v)[8]) {
  uint32_t r[8];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(addr));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&v)[4]) {
  uint32_t r[4];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(r[i]);
}
__device__ __forceinline__ void tmem_ld(uint32_t addr, float (&v)[2]) {
  uint32_t r[2];
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x2.b32 {%0,%1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(addr));
  v[0] = __uint_as_float(r[0]);
  v[1] = __uint_as_float(r[1]);
}
// waits for this thread's tmem loads; the loaded values pass through, so that none is used before
template <int W>
__device__ __forceinline__ void tmem_wait(float (&v)[W]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int i = 0; i < W; ++i) asm volatile("" : "+f"(v[i]));
}

// 16 columns of this warp's 32 lanes; tmem_stored waits for this thread's stores
__device__ __forceinline__ void tmem_st(uint32_t addr, const float (&v)[16]) {
  uint32_t r[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(v[i]);
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
          addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// One thread of the warp.  (The compiler then knows that what follows runs in one thread: products and
// copies take their operands from uniform registers, and with `lane == 0` in its place each cost over 100 clocks.)
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap* m, int x, int y, uint64_t* bar,
                                       uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
      "[%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(m), "r"(x), "r"(y), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const CUtensorMap* m, int x, int y, int z, uint64_t* bar,
                                       uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
      "[%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(m), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}
// four rows of a matrix, one under the other; a row index behind the last one reads zeros
__device__ __forceinline__ void tma_rows4(uint32_t dst, const CUtensorMap* m, int x, int r0, int r1, int r2, int r3,
                                          uint64_t* bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes.L2::cache_hint [%0], "
      "[%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(dst),
      "l"(m), "r"(x), "r"(r0), "r"(r1), "r"(r2), "r"(r3), "r"(smem_addr(bar)), "l"(policy)
      : "memory");
}
// A CTA pair's products (cta_group::2): both CTAs' copies count on the first one's barrier, one thread of the
// first CTA issues them, and their completion arrives at both.
__device__ __forceinline__ void tma_2d_pair(uint32_t dst, const CUtensorMap* m, int x, int y, uint32_t bar,
                                            uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint "
      "[%0], [%1, {%2, %3}], [%4], %5;" ::"r"(dst),
      "l"(m), "r"(x), "r"(y), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void mma_f16_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t desc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(desc), "r"(add)
      : "memory");
}
// rank: of the pair's first CTA in its cluster
__device__ __forceinline__ void mma_commit_pair(uint64_t* bar, int rank = 0) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_addr(bar)),
      "h"((uint16_t)(3 << rank))
      : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t* at, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(at)), "r"(cols)
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free_pair(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols) : "memory");
}
// a box into L2 alone
__device__ __forceinline__ void tma_prefetch_3d(const CUtensorMap* m, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(m), "r"(x), "r"(y), "r"(z)
               : "memory");
}
__device__ __forceinline__ void tma_prefetch_map(const CUtensorMap* m) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(m) : "memory");
}
__device__ __forceinline__ uint64_t policy_evict_normal() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// ---------------------------------------------------------------------------
// clusters
// ---------------------------------------------------------------------------
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// the same shared-memory address in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void peer_arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// 16 bytes into a CTA of the cluster, counted on that CTA's barrier
__device__ __forceinline__ void peer_store(uint32_t to, const float* v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
               "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
               "r"(__float_as_uint(v[3])), "r"(bar)
               : "memory");
}
// ... and not counted
__device__ __forceinline__ void peer_store(uint32_t to, const float* v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to), "r"(__float_as_uint(v[0])),
               "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])), "r"(__float_as_uint(v[3]))
               : "memory");
}
__device__ __forceinline__ bool cluster_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, 1000000;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// ---------------------------------------------------------------------------
// 16-bit values of either type
// ---------------------------------------------------------------------------
__device__ __forceinline__ float ld16(const void* p, size_t i, int bf16) {
  const unsigned short b = reinterpret_cast<const unsigned short*>(p)[i];
  return bf16 ? __uint_as_float((uint32_t)b << 16) : __half2float(__ushort_as_half(b));
}
__device__ __forceinline__ unsigned short to16(float v, int bf16) {
  return bf16 ? __bfloat16_as_ushort(__float2bfloat16_rn(v)) : __half_as_ushort(__float2half_rn(v));
}
__device__ __forceinline__ float from16(unsigned short b, int bf16) {
  return bf16 ? __uint_as_float((uint32_t)b << 16) : __half2float(__ushort_as_half(b));
}

// ---------------------------------------------------------------------------
// the ring of stages and the barriers of a CTA
// ---------------------------------------------------------------------------
struct DenseBars {
  uint64_t full[kDnMaxStages];   // TMA bytes of a stage have come
  uint64_t empty[kDnMaxStages];  // its products are done
  uint64_t tfull[2];             // a tile's sums are in TMEM
  uint64_t tempty[2];            // ... and have been read
  uint64_t drain;                // on an abort: the products in flight
  uint64_t xready, xfull;        // linear: the cluster's stages are free; its partial sums have come
  uint32_t tmem;
  int abort;
  uint32_t tries;                // rounds of a wait, kWaitTries but for diagnostics
  int last;
};

// Whether a phase of a barrier is over, without waiting for it.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_addr(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ bool dn_aborted(const DenseBars* b) { return *reinterpret_cast<const volatile int*>(&b->abort); }

// Bounded wait for a phase of a barrier; false when the time is over or another warp gave up.
__device__ __forceinline__ bool dn_wait(uint64_t* bar, uint32_t parity, const DenseBars* b) {
  if (mbar_test(bar, parity)) return true;
  for (uint32_t i = 0; i < b->tries; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (dn_aborted(b)) return false;
  }
  return false;
}

// The same for a barrier that the cluster's CTAs arrive at.
__device__ __forceinline__ bool cluster_wait(uint64_t* bar, uint32_t parity, const DenseBars* b) {
  for (uint32_t i = 0; i < b->tries; ++i) {
    if (cluster_try_wait(bar, parity)) return true;
    if (dn_aborted(b)) return false;
  }
  return false;
}

// Waits for what is in flight before a CTA ends, whoever gave up.
__device__ __forceinline__ void dn_drain(uint64_t* bar, uint32_t parity, uint32_t tries) {
  for (uint32_t i = 0; i < tries && !mbar_try_wait(bar, parity); ++i) {}
}
// ... and what no barrier of this CTA counts: after an abort it has long come when this is over.
__device__ __forceinline__ void dn_settle() {
  for (int i = 0; i < 8; ++i) __nanosleep(1000000);
}

__device__ __forceinline__ void dn_fail(DenseBars* b, int* status) {
  *reinterpret_cast<volatile int*>(&b->abort) = 1;
  set_status(status, MOE_ERR_TIMEOUT);
}

// tries: rounds of a wait; epi_warps: epilogue warps that read a tile's sums; copies: arrivals at a stage's barrier
__device__ __forceinline__ void dn_init_bars(DenseBars* b, uint32_t tries, int epi_warps = kDnEpi / 32, int copies = 1) {
  for (int i = 0; i < kDnMaxStages; ++i) {
    mbar_init(&b->full[i], copies);
    mbar_init(&b->empty[i], 1);
  }
  for (int i = 0; i < 2; ++i) {
    mbar_init(&b->tfull[i], 1);
    mbar_init(&b->tempty[i], epi_warps);
  }
  mbar_init(&b->drain, 1);
  b->abort = 0;
  b->tries = tries;
  b->last = 0;
  fence_barrier_init();
}

// True in all `n` threads of a named barrier if any of them passes true.
__device__ __forceinline__ bool dn_any(int id, int n, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred pin, pout;\n\t"
      "setp.ne.u32 pin, %3, 0;\n\t"
      "barrier.red.or.pred pout, %1, %2, pin;\n\t"
      "selp.u32 %0, 1, 0, pout;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(n), "r"((uint32_t)v)
      : "memory");
  __syncwarp();
  return r != 0;
}

// Counts the shares done of a split tile: true in every epilogue thread of the CTA whose share came
// last.  The barrier orders the CTA's stores of its partial sums before the count, whose release
// publishes them; the count's acquire and the second barrier order the reads that follow.
__device__ __forceinline__ bool dn_last_share(unsigned* cnt, int parts, DenseBars* b, int etid) {
  __syncwarp();
  named_barrier(1, kDnEpi);
  if (etid == 0) {
    unsigned old;
    asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(old) : "l"(cnt) : "memory");
    b->last = old == (unsigned)(parts - 1);
    if (b->last) *cnt = 0u;  // zero again for the next call
  }
  named_barrier(1, kDnEpi);
  return b->last != 0;
}

// g[i], u[i] = the sums over a split tile's shares, in order, of from[share * stride + i * 128] and of what lies
// `second` behind it, for i < n.  32 loads are in flight together: few tokens, many shares at a time.
template <int W>
__device__ __forceinline__ void sum_shares(const float* from, size_t second, size_t stride, int parts, int n,
                                           float (&g)[W], float (&u)[W]) {
  constexpr int U = 16 / W;
#pragma unroll
  for (int i = 0; i < W; ++i) g[i] = u[i] = 0.f;
#pragma unroll 1
  for (int s = 0; s < parts; s += U) {
    float tg[U][W], tu[U][W];
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        const bool on = s + j < parts && i < n;
        tg[j][i] = on ? __ldcg(from + (s + j) * stride + i * 128) : 0.f;
        tu[j][i] = on ? __ldcg(from + (s + j) * stride + second + i * 128) : 0.f;
      }
#pragma unroll
    for (int j = 0; j < U; ++j)
#pragma unroll
      for (int i = 0; i < W; ++i) {
        g[i] += tg[j][i];
        u[i] += tu[j][i];
      }
  }
}

// One stage's products of both 128-feature tiles, the second one `second` bytes behind the first (or, with `both`
// false, of the first alone).  The k steps of an
// operand are 32 bytes apart along its rows, 2048 across them: 2 and 128 of the descriptor's units.
// PAIR: of both CTAs of a pair.
template <bool PAIR = false>
__device__ __forceinline__ void dn_stage_products(uint32_t a, uint32_t b, uint32_t d0, uint32_t d1, uint32_t desc,
                                                  bool a_mn, bool first, bool both = true,
                                                  uint32_t second = kDnBytesA / 2) {
  const uint64_t ad = smem_desc(a, a_mn ? 8192 : 16), bd = smem_desc(b, 16);
  const uint32_t step = a_mn ? 128 : 2;
#pragma unroll
  for (int ks = 0; ks < kDnChunk / 16; ++ks) {
    const uint32_t add = !(first && ks == 0);
    if constexpr (PAIR) {
      mma_f16_pair(d0, ad + ks * step, bd + ks * 2, desc, add);
      if (both) mma_f16_pair(d1, ad + (second >> 4) + ks * step, bd + ks * 2, desc, add);
    } else {
      mma_f16(d0, ad + ks * step, bd + ks * 2, desc, add);
      if (both) mma_f16(d1, ad + (second >> 4) + ks * step, bd + ks * 2, desc, add);
    }
  }
}

// ---------------------------------------------------------------------------
// host: tensor maps
// ---------------------------------------------------------------------------
// A map of a [z][rows][cols] 16-bit array (row stride and z stride in elements) whose box is
// 64 columns by box_rows rows; out-of-range elements read as zeros.  z = 0: a plain matrix.
cudaError_t dense_map(CUtensorMap* m, const void* base, int bf16, uint64_t cols, uint64_t rows, uint64_t row_stride,
                      uint64_t z, uint64_t z_stride, uint32_t box_rows);
// A map of a dense [rows][cols] array of bytes (cols a multiple of 16) whose box is 128 columns by box_rows rows.
cudaError_t int8_map(CUtensorMap* m, const void* base, uint64_t cols, uint64_t rows, uint32_t box_rows);

}  // namespace sesg
