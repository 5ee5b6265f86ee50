// Which tile the products of an 8-bit head take (host arithmetic only, also compiled by itself in the tests).
#pragma once

#include "xent_plan.hpp"

namespace spec {

// Tiles of `bm` tokens by `bn` rows; a workgroup's waves and the steps of its pipeline are the kernel's.  `slots` of
// them fit the chip at once.  A step (a block of 128 of k) takes `full` microseconds where the chip is full of them
// and `single` where there is one per CU at most, or as long as its part of the weight takes from memory; a
// workgroup starts and stores in `ends`.  Measured in one run, bf16 logits, us with the launch:
//                          256x256 256x128 128x128 128x64 128x32 64x64 64x32
//   16 x   2048, d = 16384     155      91      83     54     49    36    30
//  256 x   4096, d = 16384     157      92      88     60     54    37    38
//  300 x  20011, d =  1024      17      13      12     18      -     -     -
//  512 x  16384, d =  4096      44      35      37     60     94    58    72
//  512 x  32768, d =  4096      65      73      81    115    181   122   147
//    1 x 151936, d =  4096       -       -       -    110    110   113   115
//   17 x 151936, d =  4096       -       -       -    116    116   119   119
//   64 x 151936, d =  4096       -       -       -    122    162   138   157
//  128 x 151936, d =  4096     185     154     167    182      -     -     -
//  256 x 151936, d =  4096     198     202     238    290      -     -     -
//  2048 x 151936, d = 4096    1187       -       -      -      -     -     -
// The model gives the order, not the times: it has 103 us for the 116 of 17 rows, where the weight comes from memory,
// 170 for the 198 of 256, and 145 and 118 for the 157 and 154 that 64 rows by 64 x 32 and 128 by 256 x 128 take; its picks
// are within 4 % of the best above.  128 x 64 and 128 x 32 read the weight past the caches and are for at most as many
// rows.  fp32 logits, whose products take twice the time, have no tile of 256.
struct LogitTile {
  int bm, bn, slots;
  double full, single, ends;
};

enum { kL256x256 = 0, kL256x128 = 1, kL128x128 = 2, kL128x64 = 3, kL128x32 = 4, kL64x64 = 5, kL64x32 = 6, kLogitTiles = 7 };

inline LogitTile logit_tile(int t, bool f32) {
  constexpr LogitTile bf16[kLogitTiles] = {{256, 256, 256, 1.65, 1.25, 8}, {256, 128, 256, 1.1, 0.70, 5},
                                           {128, 128, 512, 1.35, 0.65, 4}, {128, 64, 512, 0.85, 0.45, 3},
                                           {128, 32, 512, 0.72, 0.42, 3},  {64, 64, 512, 0.50, 0.275, 3},
                                           {64, 32, 768, 0.60, 0.26, 3}};
  constexpr LogitTile fp32[kLogitTiles] = {{256, 256, 0, 0, 0, 0},        {256, 128, 0, 0, 0, 0},
                                           {128, 128, 512, 1.85, 1.02, 4}, {128, 64, 512, 1.2, 0.66, 3},
                                           {128, 32, 512, 0.86, 0.52, 3},  {64, 64, 512, 0.70, 0.47, 3},
                                           {64, 32, 768, 0.70, 0.47, 3}};
  return f32 ? fp32[t] : bf16[t];
}

inline long long logit_work_items(int t, int N, int V) {
  constexpr int threads[kLogitTiles] = {512, 512, 256, 256, 256, 256, 128};
  const LogitTile p = logit_tile(t, false);
  return (long long)ceil_div(V, p.bm) * ceil_div(N, p.bn) * threads[t];
}

inline double logit_us(int t, bool f32, int N, int V, int d) {
  const LogitTile p = logit_tile(t, f32);
  const long long tj = ceil_div(N, p.bn), tiles = ceil_div(V, p.bm) * tj, rounds = tiles / p.slots, rest = tiles % p.slots;
  const double share = tj < 8 ? (double)tj : 8.0;   // tiles that share a strip of the weight in a cache
  auto step = [&](long long k) {
    const double memory = k * p.bm * 128.0 / share / 6.7e6, work = k > (p.slots > 256 ? 256 : 128) ? p.full : p.single;
    return memory > work ? memory : work;
  };
  const double steps = ceil_div(d, 128);
  return rounds * (steps * step(p.slots) + p.ends) + (rest ? steps * step(rest) + p.ends : 0.0);
}

inline int pick_logit_tile(bool f32, int N, int V, int d) {
  int best = -1;
  double us = 0;
  for (int t : {kL64x32, kL64x64, kL128x32, kL128x64, kL128x128, kL256x128, kL256x256}) {
    if (logit_tile(t, f32).slots == 0 || (t == kL128x32 && N > 32) || (t == kL128x64 && N > 64)) continue;
    const double c = logit_us(t, f32, N, V, d);
    if (best < 0 || c < us) {
      best = t;
      us = c;
    }
  }
  return best;
}

}  // namespace spec
