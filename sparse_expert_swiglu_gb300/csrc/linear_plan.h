// The tile, stages and cluster of a product (linear.cu), by its sizes alone.
#pragma once

#include <initializer_list>

#include "dense_plan.h"

namespace sesg {

struct LinearPlan {
  int M = -1, N = 0, K = 0, gated = 0, kn = 0, plain = 0, f32 = 0, sms = 0, room = 0;  // what it is for
  int by_token = 0;  // linear_pair_kernel
  int P = 1, NT = 0, MT = 0, rows = 0, both = 0, wide = 1, S = 0, T = 0;
};

constexpr int kFewTokens = 32;
constexpr int kTogether = 8;  // token tiles that go through all features together

// Clusters of S CTAs that fit the GPU at once, of at most one CTA per SM (152 SMs: 76, 36 and 15; the SMs of a
// cluster lie in one part of the chip).  For the model alone: where fewer fit, a call takes longer and gives the same.
inline int clusters(int S, int sms) { return S == 1 ? sms : S == 2 ? sms / 2 : S == 4 ? sms / 4 - 2 : sms / 8 - 4; }

// Bytes of a cluster's partial sums in one CTA.
inline int linear_sum_bytes(const LinearPlan& l, int M, bool gated) {
  return (gated ? 2 : 1) * (((M < l.NT ? M : l.NT) + 3) / 4) * 4096;
}

// Stages of a CTA, and whether the partial sums have memory behind them (up to 16 KB).  room: bytes for both.
inline int linear_stages(const LinearPlan& l, int M, bool gated, int room, bool& own_x) {
  const int stage = l.wide * ((l.both ? kDnBytesA : kDnBytesA / 2) + l.NT / l.P * 128), sums = linear_sum_bytes(l, M, gated);
  own_x = l.S > 1 && sums <= 16384;
  const int n = (room - (own_x ? sums : 0)) / stage;
  return n > kDnMaxStages ? kDnMaxStages : n;
}

// Accumulators of a product.  The tensor core cuts off what its fp32 additions cannot hold: an accumulator that adds up
// n steps of 16 k loses up to (2/3) n 2^-24 of its sum, always towards zero (measured at 4096 k: 4.4e-6 of the result).
// So stages of an fp32 result go round up to eight accumulators where TMEM has the columns, none takes more than 1024 k
// (16-bit results: 16384), and where that does not cover a tile's k, they start anew, in two sets by turns, and the
// epilogue's warps add the rounds up in registers.
struct LinearSums {
  int groups, bufs;  // accumulators of a product; sets of them, so that one can be read while the next is filled
  int per, keep;     // stages of a round; whether there are several
  int cols;          // TMEM columns of all
};
constexpr int sum_chunks(bool f32) { return f32 ? 16 : 256; }  // of 64 k, that one accumulator takes

// False: a warp's registers do not hold its share of the sums (128 columns).
inline bool linear_sums(const LinearPlan& l, int K, bool f32, LinearSums& s) {
  const int KC = ((K + kDnChunk - 1) / kDnChunk + l.wide - 1) / l.wide, share = (KC + l.S - 1) / l.S;
  const int cols = (l.both ? 2 : 1) * l.NT, most = sum_chunks(f32) / l.wide;
  s.keep = 0;
  s.bufs = cols <= 256 && l.S == 1 && l.T > l.sms / l.P ? 2 : 1;  // two where a CTA has more than one tile
  s.groups = 1;
  while (f32 && s.groups < 8 && 2 * s.groups * cols * s.bufs <= 512) s.groups *= 2;
  s.per = share;
  if (share > s.groups * most) {
    s.keep = 1;
    s.groups = 1;
    s.bufs = 2;
    s.per = most;
  }
  s.cols = s.groups * cols * s.bufs;
  return !s.keep || cols <= 256;
}

// The tile and the cluster with the least time by a model in SM clocks.  Its terms, as measured (GB300,
// 1.9 GHz):
//   a call costs 7000 whatever it does (256 x 512, one token: 3.8 us);
//   an SM takes 62 bytes a clock from L2 (tiles of 128 x 128: 32 KB in 516 clocks), all SMs together
//   3550 out of HBM, and where both are needed the lesser adds 0.15 of itself; rows that do not start
//   on a line of 128 bytes take 1.35 times as long out of L2, and 1.8 times where they start inside a sector of
//   32 (333 x 1024 by 128 x 32: K = 1000 8.9 us, K = 1024 7.0; 1017 x 7760 gated, K = 3280, pairs with 64 and 128 columns:
//   537 and 704 clocks a stage instead of 370 and 650);
//   a stage's bytes start to come 1950 after they are asked for (4096 x 4096, one token, 16 KB stages: six of them
//   run at 383 clocks each, three 32 KB ones at 831), and a stage costs its issuing threads 270 and for
//   each 64 k 155 + 3 NT (2048 x 2048, 16 tokens: 64 / 128 / 256 k a stage 11.9 / 9.5 / 8.3 us), and 60 more
//   where its rows are shorter boxes;
//   a product of 128 x NT x 16 takes NT / 2, and a quarter more with all SMs at it (the clock drops);
//   joining a cluster's sums 3300 and 48 for each token and product; a tile's epilogue 18 for
//   each token and product and, but for the last, 1500; it runs under the next tile's products where TMEM holds both;
//   a CTA pair's stage 650 with 256 columns, and 27 a column for its last epilogue, and HBM
//   adds 0.25 of the weights' time (2048 x 14336 gated, K = 4096: 275 us against the model's 279; one CTA a
//   tile 321; 300 tokens 80 and 80); 90 a column for the others,
//   which run under the next tile's products (384 x 7808 gated, GELU, K = 120: 7200 for 64 columns); 6 a column for a
//   round of sums that is added up, under the next round's products.
inline LinearPlan make_plan(int M, int N, int K, bool gated, bool kn, bool plain, bool f32, int sms, int room) {
  LinearPlan best;
  double best_t = 1e30;
  const int chunks = (K + kDnChunk - 1) / kDnChunk, mats = gated ? 2 : 1;
  const double w_bytes = 2.0 * mats * N * K, hbm = 3550;
  auto keep = [&](const LinearPlan& l, double t) {
    if (t < best_t) {
      best_t = t;
      best = l;
    }
  };
  auto slow = [](int row) { return row % 64 == 0 ? 1.0 : row % 16 == 0 ? 1.35 : 1.8; };
  const double slow_x = slow(K), slow_w = slow(kn ? N : K);
  LinearPlan l;
  l.sms = sms;
  if (plain && N % 8 == 0 && M > 64) {
    // [K][N] weights come in boxes of 64 columns: narrower tiles would start inside a line (2048 x 4096, K = 14336: 148 us
    // with 128 columns, 186 with 112, which would fill two whole waves; [N][K] 176 and 158)
    for (int rows = 64; rows <= kDnHalf; rows += gated || kn ? 64 : 16) {
      const int width = gated ? rows : 2 * rows, MT = (M + 255) / 256;
      const long long T = (long long)MT * ((N + width - 1) / width);
      if (T > (1 << 30) || (!gated && N <= rows)) continue;
      l.by_token = 1;
      l.S = 1;
      l.T = (int)T;
      l.MT = MT;
      l.rows = rows;
      const double waves = (double)((T + sms / 2 - 1) / (sms / 2)), chunk = 650.0 * rows / kDnHalf;
      const double l2 = (kDnHalf * slow_x + rows * slow_w) * 128 / 62;
      const double products = chunks * (chunk > l2 ? chunk : l2), epi = 90.0 * rows;
      // rounds are added up under the next one's products
      const double rounds = chunks > sum_chunks(f32) ? chunks / sum_chunks(f32) * 6.0 * rows : 0;
      const double t = waves * (products > epi + rounds ? products : epi + rounds);
      const double mem = w_bytes / hbm;
      keep(l, 7000 + 27.0 * rows + (t > mem ? t + 0.25 * mem : mem + 0.25 * t));
    }
  }
  auto consider = [&](int P, int NT, int rows, int both, int wide, int S) {
    l.by_token = 0;
    l.P = P;
    l.wide = wide;
    const int KC = (chunks + wide - 1) / wide;
    l.MT = (M + NT - 1) / NT;
    l.NT = ((M + l.MT - 1) / l.MT + 16 * P - 1) / (16 * P) * 16 * P;
    l.rows = rows;
    l.both = both;
    l.S = S;
    const int width = P * (gated || !both ? rows : 2 * rows), fit = clusters(P * S, sms), toks = l.NT / P;
    const long long T = (long long)((N + width - 1) / width) * l.MT;
    if (wide / 2 >= chunks) return;  // half of the stage would do
    if (T > (1 << 30) || (both && !gated && N <= rows) || (P > 1 && N <= width / 2) || (S > 1 && (T > fit || S > KC))) return;
    l.T = (int)T;
    bool own_x;
    LinearSums sums;
    if (!linear_sums(l, K, f32, sums)) return;
    const int stage = wide * ((both ? kDnBytesA : kDnBytesA / 2) + toks * 128);
    const int stages = linear_stages(l, M, gated, room, own_x);
    if (stages < 2 || (S > 1 && !own_x && linear_sum_bytes(l, M, gated) > stages * stage)) return;
    const double waves = (double)((T + fit - 1) / fit), active = (double)(T < fit ? T : fit) * S * P;
    const double load = wide * ((both ? 2 : 1) * rows + toks) * 128.0, w_load = load - wide * toks * 128.0;
    const double mma = wide * (both ? 2 : 1) * 4 * 1.25 * l.NT / 2;
    const double l2 = (w_load * slow_w + (load - w_load) * slow_x) / 62;
    // weights that several token tiles share come out of HBM little more than once: those tiles run together (32 x 4096 x
    // 4096 as 16 + 16 tokens 13.2 us, as 32 11.3)
    const double mem = w_load * active / hbm / (1 + 0.65 * ((l.MT < kTogether ? l.MT : kTogether) - 1));
    double chunk = l2 > mem ? l2 + 0.15 * mem : mem + 0.15 * l2;
    for (const double least : {mma, (1950 + l2 + mma) / stages, 270 + wide * (155 + 3.0 * toks)})
      if (chunk < least) chunk = least;
    if (rows < kDnHalf) chunk += 60 * wide;
    const double last = 18.0 * l.NT * (both ? 2 : 1), epi = 1500 + last;
    const double products = (((KC + S - 1) / S) * chunk + (l2 + mma) / 2) * (P == 2 ? 1.05 : 1);
    double t = S > 1 ? products + 3300 + 48.0 * l.NT * (both ? 2 : 1)
               : l.NT * (both ? 2 : 1) <= 256 ? waves * (products > epi ? products : epi) + last
                                              : waves * (products + epi) - 1500;
    if (t < w_bytes / hbm) t = w_bytes / hbm;
    t *= wide == 1 ? 1 : wide == 2 ? 0.98 : 0.96;  // 216 KB in flight instead of 147
    keep(l, 7000 + t);
  };
  const int top = M < 256 ? (M + 15) / 16 * 16 : 256;
  for (int both = gated ? 1 : 0; both < 2; ++both)
    for (int rows = both && !gated ? kDnHalf : kn ? 64 : 32; rows <= kDnHalf && (rows < N + 64 || rows <= 64); rows += kn ? 64 : 32)
      for (int NT = 16; NT <= top; NT += 16)
        for (int S = 1; S <= 8; S *= 2)
          for (int wide = 1; wide <= 4; wide *= 2) {
            consider(1, NT, rows, both, wide, S);
            if (M > 64 && NT % 32 == 0 && S <= 4) consider(2, NT, rows, both, wide, S);
          }
  best.M = M;
  best.N = N;
  best.K = K;
  best.gated = gated;
  best.kn = kn;
  best.plain = plain;
  best.f32 = f32;
  best.sms = sms;
  best.room = room;
  return best;
}

// The plan goes by the sizes alone.  A thread keeps the plans of the sizes that it used last, since a model's calls come
// again with every token: 16 sets of 8, of which a new plan takes the place of the one that was asked for longest
// ago.  The sizes are mixed one into the other: two calls with the same M (the products of an expert) must not fall into
// one set for every M.
inline const LinearPlan& linear_plan(int M, int N, int K, bool gated, bool kn, bool plain, bool f32, int sms, int room) {
  constexpr int kSets = 16, kWays = 8;
  struct Kept {
    LinearPlan plan[kWays];
    uint64_t used[kWays] = {};
  };
  static thread_local Kept sets[kSets];
  static thread_local uint64_t now = 0;
  uint64_t h = 0;
  for (const int v : {M, N, K, (int)f32 * 8 + (int)gated * 4 + (int)kn * 2 + (int)plain}) {
    h = (h ^ (uint32_t)v) * 0x9E3779B97F4A7C15ull;
    h ^= h >> 29;
  }
  Kept& s = sets[h % kSets];
  int oldest = 0;
  for (int i = 0; i < kWays; ++i) {
    const LinearPlan& l = s.plan[i];
    if (l.M == M && l.N == N && l.K == K && l.gated == gated && l.kn == kn && l.plain == plain && l.f32 == f32 &&
        l.sms == sms && l.room == room) {
      s.used[i] = ++now;
      return l;
    }
    if (s.used[i] < s.used[oldest]) oldest = i;
  }
  s.plan[oldest] = make_plan(M, N, K, gated, kn, plain, f32, sms, room);
  s.used[oldest] = ++now;
  return s.plan[oldest];
}

}  // namespace sesg
