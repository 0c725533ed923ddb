// The tile, stages and cluster of a product of 8-bit integers (linear_int8_tiles.cu) and the threads of the quantiser
// (quantize.cu), by their sizes alone.
#pragma once

#include "linear_plan.h"

namespace sesg {

constexpr int kI8Threads = 640;      // warps: 0 TMA, 1 products, 2 TMEM, 4-11 integers to fp16, 12-19 epilogue
constexpr int kI8Chunk = 128;        // k of a stage: 128 bytes of a row of w, 256 of a token
constexpr int kI8Round = 8;          // stages that one accumulator takes: 1024 products of at most 2^14 are exact in fp32
constexpr int kI8Cols = 192;         // TMEM columns of one set of accumulators, at most; there are two
constexpr int kI8MaxSlots = 8;       // of 64 k (32 columns) with more than 128 tokens in a tile, else 128 k: rows of w as fp16
constexpr int kI8Halves = 16384;     // bytes: what epilogue warps exchange with w_mul

// With more than 64 tokens in a tile the warps share out the registers that a block is launched with: warps 0-3, those that
// convert, those of the epilogue.  Shares beyond those would wait forever.  Registers are allotted in units of 8 a thread.
constexpr int kI8RegsIssue = 48, kI8RegsConvert = 72, kI8RegsEpilogue = 144;
inline bool int8_registers_fit(int a_thread) {
  return (a_thread + 7) / 8 * 8 * kI8Threads >= 128 * kI8RegsIssue + 256 * kI8RegsConvert + 256 * kI8RegsEpilogue;
}

struct Int8Plan {
  int P = 1;       // CTAs that run one product (cta_group::2 with 2)
  int S = 0;       // shares of k: a cluster has P S CTAs
  int rows = 0;    // features of a CTA's tile: up to 128, with w_mul 64
  int NT = 0, MT = 0, T = 0;  // tokens of a tile, token tiles, tiles
  int blocks = 0;  // blocks of 16 columns that an epilogue warp adds up: 1, 2, 4 or 6
  int stages = 0, slots = 0;
};

// Shared memory behind the stages and barriers: the tokens' scales, one array for each epilogue warp, and those halves.
inline int int8_extra_bytes(bool gated) { return kI8Cols / 2 * 8 * 4 + (gated ? kI8Halves : 0); }
inline int int8_stage_bytes(const Int8Plan& l) { return 128 * kI8Chunk + l.NT / l.P * kI8Chunk * 2; }
// Bytes of a cluster's partial sums in one CTA: 8 warps' tokens, 128 bytes each.
inline int int8_sum_bytes(const Int8Plan& l) { return (l.NT + 31) / 32 * 16 * 8 * 128; }

// The tile and the cluster with the least time by a model in SM clocks (at 1.9 GHz).  Its terms are fitted to measured times
// under every tile and cluster that a size allows (190 of 17 sizes, the join's again to 258 of 22, 16 to 2048 tokens; the
// errors' root mean square is 6 and 9 %).  What it chooses of the 258 is in the mean 0.5 % slower than the fastest, 10 % at
// worst (40 tokens of 2 x 2048 x 2048: 9.95 us, 9.03 in clusters of four):
//   a call costs 9700 whatever it does, its tokens' kernel included, and 40 for each token of a tile;
//   an SM takes 57 bytes a clock from L2, all SMs together 3200 out of HBM, to which token tiles that run together add little;
//   a stage takes 6.8 for each token in one CTA, 5.6 in a pair, and never less than 470 (600), which its barriers take;
//   filling the ring 1600 a tile; the epilogue 48 for each token and round (with w_mul 13 more a token), under the next
//   tile's products; joining a cluster's sums 3000 and 28 for each token.
inline Int8Plan make_int8_plan(int M, int N, int K, bool gated, int sms, int room) {
  const int feats = gated ? 64 : 128, KC = (K + kI8Chunk - 1) / kI8Chunk;
  Int8Plan best;
  double best_t = 1e300;
  for (int P = 1; P <= 2; ++P) {
    if (P == 2 && (M <= 96 || N <= feats)) continue;
    for (int NT = 32; NT <= kI8Cols; NT += 32) {
      if (NT > 32 && NT - 32 >= M) break;  // the tile before holds them all
      Int8Plan l;
      l.P = P;
      l.MT = (M + NT - 1) / NT;
      if (M <= 16 && P == 1) l.NT = 16;
      else l.NT = ((M + l.MT - 1) / l.MT + 31) / 32 * 32;
      const int tb = (l.NT + 31) / 32;
      l.blocks = P == 1 && tb <= 2 ? tb : tb <= 4 ? 4 : 6;
      const int free_slots = (512 - 2 * l.NT) / (l.blocks == 6 ? 32 : 64);
      l.slots = free_slots < kI8MaxSlots ? free_slots : kI8MaxSlots;
      const int stage = int8_stage_bytes(l);
      l.stages = room / stage < kDnMaxStages ? room / stage : kDnMaxStages;
      if (l.blocks <= 2 && l.stages > l.slots) l.stages = l.slots;  // a slot is free when its stage is
      l.stages &= ~1;  // two sets of warps take turns, and a stage must always be the same set's
      if (l.stages < 2) continue;
      for (int S = 1; S * P <= 8; S *= 2) {
        l.S = S;
        const int fit = clusters(P * S, sms);
        // Where w's bytes are the bound: as few features as fill the last wave (whole 32-byte sectors of a token's row).
        const long long most = (long long)((N + feats * P - 1) / (feats * P)) * l.MT;
        if (most > (1 << 30) || fit < 1) continue;
        const long long waves = (most + fit - 1) / fit, ft = waves * fit / l.MT;
        l.rows = l.MT > 1 ? feats : (int)((N + ft * P - 1) / (ft * P) + 15) / 16 * 16;
        if (l.rows > feats) l.rows = feats;
        l.T = (N + l.rows * P - 1) / (l.rows * P) * l.MT;
        if (S > 1 && (l.T > fit || S > KC || int8_sum_bytes(l) > l.stages * stage)) continue;
        const double active = (double)(l.T < fit ? l.T : fit) * S * P;
        const double bytes = (gated ? 2 : 1) * l.rows * 128.0, load = bytes + l.NT / P * 256.0;
        const double mem = bytes * active / 3200 / (1 + 0.5 * ((l.MT < kTogether ? l.MT : kTogether) - 1));
        double stage_t = load / 57;
        for (const double least : {mem, (P == 1 ? 6.8 : 5.6) * l.NT, P == 1 ? 470.0 : 600.0})
          if (stage_t < least) stage_t = least;
        const int share = (KC + S - 1) / S;
        const double tile = share * stage_t + 1600, epi = l.NT * (48.0 * ((share + kI8Round - 1) / kI8Round) + (gated ? 13 : 0));
        const double t = waves * (tile > epi ? tile : epi) + 40.0 * l.NT + (S > 1 ? 3000 + 28.0 * l.NT : 0);
        if (t < best_t) {
          best_t = t;
          best = l;
        }
      }
    }
  }
  return best;
}

// Threads of the quantiser for each row.  Many rows: 8 loads of 16 bytes for each thread, so that enough bytes are in flight
// beside the rows that wait or round.  Few (two a SM): 2, so that a row is over soon.
inline int quantize_threads(int rows, int K, bool f32, int sms) {
  const int keep = rows <= 2 * sms ? 2 : f32 ? 4 : 8;  // vectors of eight elements, which are two loads in fp32
  int T = 32;
  while (T < 1024 && T * keep < K / 8) T *= 2;
  return T;
}

// A thread keeps the plans of the sizes that it used last, which a model's calls come back to: 64 of them, by their mixed
// sizes.
inline const Int8Plan& int8_plan(int M, int N, int K, bool gated, int sms, int room) {
  struct Kept {
    int key[6] = {-1, 0, 0, 0, 0, 0};
    Int8Plan plan;
  };
  static thread_local Kept kept[64];
  const int key[6] = {M, N, K, (int)gated, sms, room};
  uint64_t h = 0;
  for (const int v : key) {
    h = (h ^ (uint32_t)v) * 0x9E3779B97F4A7C15ull;
    h ^= h >> 29;
  }
  Kept& k = kept[h % 64];
  bool same = true;
  for (int i = 0; i < 6; ++i) same = same && k.key[i] == key[i];
  if (!same) {
    k.plan = make_int8_plan(M, N, K, gated, sms, room);
    for (int i = 0; i < 6; ++i) k.key[i] = key[i];
  }
  return k.plan;
}

}  // namespace sesg
