// The tiles and the workspace of a dense layer (dense_layer.cu), by its sizes alone.
#pragma once

#include "dense_plan.h"

namespace sesg {

constexpr int kDenseMaxTok = 64;
constexpr int kPartFloats = 2 * kDenseMaxTok * kDnHalf;
constexpr int kFewTok = 8;                       // up to here every CTA chooses the experts itself

// Groups of 8 slots that the active experts' tokens fill, at most.
inline int max_groups(int B, int E, int k, int ns) {
  const int pairs = B * k, active = E < pairs ? E : pairs;  // one for each active expert, another for every 8 more pairs
  return active + (pairs - active) / 8 + ns * ((B + 7) / 8);
}

// Rows of the second phase's sums: one for each (token, expert) pair; of a few tokens one for each slot.
inline int sum_rows(int B, int E, int k, int ns) {
  return B <= kFewTok ? 8 * max_groups(B, E, k, ns) : B * (k + ns);
}

struct LayerPlan {
  int B = -1, d, f, E, k, ns, sms;
  int groups, slices, grid, rows, wide, early;
  size_t logits, top_idx, top_w, h, part, yrow, ysq, ysum, total;
};

constexpr int kSmem = 232448;  // that the plan reckons with

inline int layer_a_bytes(int rows, int wide) { return wide * 2 * rows * 128 > kDnBytesA ? wide * 2 * rows * 128 : kDnBytesA; }

inline int layer_stages(int B, int rows, int wide, int slots, int misc, int smem) {
  const int n = (smem - 1024 - misc - slots) / (layer_a_bytes(rows, wide) + (B + 7) / 8 * 16 * 128);
  return n > kDnMaxStages ? kDnMaxStages : n;
}

// The plan goes by the sizes alone (misc and head: bytes of the kernel's lists and of the workspace's head); a thread
// keeps the last one, since a program calls with the same sizes again and again.
inline const LayerPlan& layer_plan(int B, int d, int f, int E, int k, int ns, int sms, int misc, size_t head) {
  static thread_local LayerPlan l;
  if (l.B == B && l.d == d && l.f == f && l.E == E && l.k == k && l.ns == ns && l.sms == sms) return l;
  l.B = B;
  l.d = d;
  l.f = f;
  l.E = E;
  l.k = k;
  l.ns = ns;
  l.sms = sms;
  l.grid = sms;
  l.groups = max_groups(B, E, k, ns);
  l.slices = B > 0 ? sms / B : 1;
  const int rows = (d + 63) / 64;  // 64 rows of the router weight at least
  if (l.slices > 16) l.slices = 16;
  // the logits of a few tokens' slices are gathered in one stage
  if (B > 0 && B <= kFewTok && l.slices > 8192 / (B * E)) l.slices = 8192 / (B * E);
  if (l.slices > rows) l.slices = rows;
  if (l.slices < 1) l.slices = 1;
  const int DT = (d + 2 * kDnHalf - 1) / (2 * kDnHalf);
  const int chunks = (d + kDnChunk - 1) / kDnChunk, KC2 = (f + kDnChunk - 1) / kDnChunk;
  const int most = E < B * k ? E : B * k;
  // Features of a tile: those with which the expected number of active experts (one token: the exact one)
  // comes nearest to whole waves, so that no tile's sums have to be joined.
  double miss = 1;
  for (int b = 0; b < B; ++b) miss *= 1 - (double)k / E;
  const int act = ns + (int)(E * (1 - miss) + 0.5);
  // The shared experts' tiles may start before the routing, which is worth 2 chunks, but are whole then: with few
  // tiles they last longer than all the others, cut into equal shares (61 tokens of 19 experts of 280 features, 8 + 2 for each:
  // 76 us with whole ones, 55 without).
  double best = 1e30;
  for (int rows = kDnHalf; rows >= 64; rows -= 8) {
    for (int first = ns > 0; first >= 0; --first) {
      const int FT = (f + rows - 1) / rows, early = first ? ns * FT : 0;
      const Sched s = Sched::make(act * FT, chunks, sms, early);
      // clocks of the slowest SM: a tile's chunks at its share of HBM, and 6 chunks' worth for joining
      const double chunk = rows / 128.0, tail = s.total ? (double)s.total / sms * chunk + 6 : 0;
      const double t = (s.dp + sms - 1) / sms * chunks * chunk + tail + (ns > 0 && !first ? 2 : 0);
      if (t < best * 0.995) {
        best = t;
        l.rows = rows;
        l.early = early;
      }
    }
  }
  // Low tiles leave much of a stage empty.  Where the stages are too few for their bytes' 2.1 us under way (an SM's share of
  // HBM brings 128 rows in 0.7), two chunks go into one (63 tokens of 6 x 1664, 72 rows: 76.8 us with one, 71.6 with two).
  l.wide = l.rows <= 80 && 3.0 / layer_stages(B, l.rows, 1, l.groups * 8, misc, kSmem) > l.rows / 128.0 ? 2 : 1;
  // the number of active experts is known on the device only: the largest need of any
  int segs1 = 0, segs2 = 0;
  const int KC1 = (chunks + l.wide - 1) / l.wide;
  const int FT = (f + l.rows - 1) / l.rows;
  for (int a = 0; a <= most; ++a) {
    const Sched s1 = Sched::make((a + ns) * FT, KC1, sms, l.early), s2 = Sched::make((a + ns) * DT, KC2, sms, 0);
    if (s1.segments() > segs1) segs1 = s1.segments();
    if (s2.segments() > segs2) segs2 = s2.segments();
  }
  size_t o = (head + 255) / 256 * 256;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = (o + bytes + 255) / 256 * 256;
    return at;
  };
  l.logits = take((size_t)B * l.slices * E * 4);
  l.top_idx = take((size_t)B * k * 4);
  l.top_w = take((size_t)B * k * 4);
  l.h = take((size_t)l.groups * 16 * f * 2);
  l.yrow = take((size_t)B * d * 4);
  l.ysq = take((size_t)B * 2 * DT * 16);
  // the second phase's sums: of whole tiles by token and expert, then the shares of cut tiles, which take the place
  // of the first phase's shares (all of those are read before any CTA has h for its second phase)
  l.ysum = take((size_t)sum_rows(B, E, k, ns) * d * 4);
  const size_t part1 = (size_t)segs1 * kPartFloats * 4, part2 = (size_t)segs2 * B * 2 * kDnHalf * 4;
  l.part = take(part1 > part2 ? part1 : part2);
  l.total = o;
  return l;
}

}  // namespace sesg
