// Sizes that the kernels on uncompressed weights and their plans share.  Host code without CUDA: the plans compile
// with any C++ compiler.
#pragma once

#include <cstddef>
#include <cstdint>

#ifdef __CUDACC__
#define SESG_HD __host__ __device__
#else
#define SESG_HD
#endif

namespace sesg {

constexpr int kDnThreads = 384;      // warps: 0 TMA, 1 products, 2 TMEM, 4-11 epilogue
constexpr int kDnEpi = 256;          // ... threads: two warps for every 32 TMEM lanes
constexpr int kDnChunk = 64;         // k per stage: 128 bytes, one swizzled row
constexpr int kDnHalf = 128;         // features of one product (TMEM lanes)
constexpr int kDnBytesA = 2 * kDnHalf * kDnChunk * 2;
constexpr int kDnMaxStages = 8;
constexpr int kDnMaxSplit = 16;      // shares of one tile along k, at most (plus a border)
constexpr int kDnMaxCtas = 1024;

// ---------------------------------------------------------------------------
// Work of CTA c of P: T tiles of KC chunks each.  Tiles below dp are whole: c, c + P, ...
// The others lie in one line of (T - dp) * KC chunks, of which CTA c takes q from c * q.
// ---------------------------------------------------------------------------
struct Sched {
  int T, KC, P, dp, q, total;
  // at least the first `whole` tiles stay whole
  SESG_HD static Sched make(int T, int KC, int P, int whole) {
    Sched s;
    s.T = T;
    s.KC = KC;
    s.P = P;
    // Joining the shares of the last tiles takes about 4 us, and a chunk 0.7 us: a last wave that leaves less
    // than that idle on average is not cut.
    const int rest = T % P;
    s.dp = (P - rest) * KC * 10 <= 57 * P ? T : T - rest;
    if (s.dp < whole) s.dp = whole;
    s.total = (T - s.dp) * KC;
    const int by_ctas = (s.total + P - 1) / P, by_split = (KC + kDnMaxSplit - 1) / kDnMaxSplit;
    s.q = by_ctas > by_split ? by_ctas : by_split;
    if (s.q < 1) s.q = 1;
    return s;
  }
  // shares of a split tile (t >= dp) and the CTA of the first one
  SESG_HD int first(int t) const { return (t - dp) * KC / q; }
  SESG_HD int parts(int t) const { return t < dp ? 1 : ((t - dp + 1) * KC - 1) / q - first(t) + 1; }
  SESG_HD int max_parts() const { return total ? (KC + q - 1) / q + 1 : 1; }
  // partial sums in the workspace: numbered along the line of shares
  SESG_HD int segments() const { return total ? (T - dp) + (total + q - 1) / q : 0; }
};

}  // namespace sesg
