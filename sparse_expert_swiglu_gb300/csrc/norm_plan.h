// The threads and CTAs of the norms around a block (residual_norm.cu), by their sizes and types alone.
#pragma once

#include <cstddef>

namespace sesg {

constexpr size_t kNormShared = 200 << 10;  // of an SM, for what comes ahead

struct NormPlan {
  bool ahead;     // a CTA goes from token to token, the next one's values come ahead
  int nv;         // vectors of 8 for each thread
  int threads, ctas;
  size_t bytes;   // shared memory of what comes ahead
};

// Ahead a thread has 2 vectors (8192 x 4096, LayerNorms and an fp32 residual, when all were timed: 73 us, with 1 81, with 4 79;
// 1000 x 8208 13.9 us, with 4 15.0), else 1, which leaves one token's barriers with the least work between (64 x 8192, RMSNorm:
// 3.1 us, with 2 4.3).  An SM holds one CTA of more than 512 threads: where there are more tokens than SMs, two smaller ones are
// faster (300 x 8192: 5.6 us, else 6.7), but for rows that need 2 vectors of 1024 threads (300 x 16384: 11.0 us, with 4 of 512
// 13.9).
//
// Which of the two: values ahead pay from about 0.6 of the tokens on that fit the chip at once (with two vectors a thread these
// are more than with one), in us without and with: 608 x 1024 2.51 and 2.66, 1702 x 1024 4.47 and 4.10, 608 x 2048 3.31 and 3.51,
// 851 x 2048 4.67 and 4.17, 400 x 4096 4.90 and 4.20 (RMSNorm); to 8 bits 608 x 2048 4.11 and 4.84, 1216 x 2048 6.99 and 6.55;
// LayerNorms and an fp32 stream 608 x 2048 5.27 and 5.71, 851 x 2048 7.72 and 7.29.  But never with fewer tokens than two a SM, and
// where one warp has a token, whose sums need no barrier, from all of them on (2553 x 256 3.18 and 3.38, 4742 x 256 5.20 and 4.37),
// to 8 bits or with an fp32 stream from 2.5 times as many (5836 x 256 6.43 and 7.31, 7296 x 256 7.82 and 7.42, 10944 x 512 13.8
// and 13.5).  Over 220 sizes and forms drawn afterwards (305 to 20000 tokens of 64 to 16384) the choice is in the mean 0.7 % slower
// than the faster form, always ahead 6 %.
inline NormPlan norm_plan(int M, int d, bool residual, bool s_f32, bool y_int8, int sms) {
  const int n = d / 8;
  NormPlan l;
  auto threads = [&](int nv) { return ((n + nv - 1) / nv + 31) / 32 * 32; };
  l.nv = 2;
  l.threads = threads(2);
  l.bytes = (size_t)2 * (residual ? s_f32 ? 3 : 2 : 1) * l.threads * 16;
  // CTAs that fit an SM at once, by threads and shared memory
  int fit = 1024 / l.threads < 24 ? 1024 / l.threads : 24;
  if (fit > (int)(kNormShared / (l.bytes + 1536))) fit = (int)(kNormShared / (l.bytes + 1536));
  const long long all = (long long)fit * sms;
  l.ahead = l.threads > 32 ? M > 2 * sms && 5LL * M > 3 * all : 2LL * M > (y_int8 || (residual && s_f32) ? 5 : 2) * all;
  l.ctas = l.ahead && M > all ? (int)all : M;
  if (!l.ahead) {
    l.nv = n > 1024 || (n > 512 && M > sms) ? 2 : 1;
    l.threads = threads(l.nv);
    l.bytes = 0;
  }
  return l;
}

}  // namespace sesg
