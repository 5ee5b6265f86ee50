// How the vocabulary head's products are cut up: tile shapes, shared tiles and pieces of the vocabulary (host
// arithmetic only, also compiled by itself in the tests).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#include "spec_verify.h"

namespace spec {

constexpr int kStepBytes = 128;   // of k per row and pipeline step

inline int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }
inline long long round_to(long long a, long long b) { return (a + b - 1) / b * b; }
inline size_t round_bytes(size_t x) { return (x + 255) & ~(size_t)255; }

// Tile shapes of the product.  bf16: 256 x 256 (8 waves, one workgroup per CU); 128 x 128 or, for rowsB of at
// most 64, 128 x 64 (4 waves, two per CU); and for kStats and kGradZ, where there are few tiles and a step
// waits for its loads, 128 x 64 with six steps in flight (one per CU) and 64 x 64 with five (two per CU).
// Loss and gradients of 348 x 717, d = 3064 by the three last shapes: 32, 24, 19.5 us and 85, 63, 55 us; of
// 1000 x 1000, d = 2048: 28, 18, 15 and 72, 60, 56; of 246 x 6727, d = 2896 (two of the smallest tiles per
// CU): 44, 29.7, 32.3.  At most 64 rows by 128 x 64 and by 64 x 64: 1 x 1000, d = 4096: 30.0, 20.8 us and 40.5,
// 35.1; 64 x 717, d = 3064: 23.0, 18.8 and 39.6, 34.7; 64 x 8000, d = 2048: 21.3, 16.0 and 57.2, 49.0; from
// some 20000 tokens on there are two 128 x 64 tiles per CU and they stay.  fp32 is bound by the matrix units (a sixteenth of the bf16 rate), so what counts is
// that every CU has its share: 128 x 64 (against 128 x 128 and 256 x 256, 200 x 20000, d = 1024: 132 -> 109 us;
// gradients of 1000 x 1000, d = 2048: 197 -> 169), or 64 x 64 (76 -> 44 us; 169 -> 135; each before the sums in
// blocks, which add 1 to 3 %).
enum { kBig = 0, kMid = 1, kThin = 2, kDeep = 3, kSmall = 4 };

inline int tile_m(int t) { return t == kBig ? 256 : t == kSmall ? 64 : 128; }
inline int tile_n(int t) { return t == kBig ? 256 : t == kMid ? 128 : 64; }
inline int strip_rows(int t) { return tile_m(t) / 2; }          // of kStats
inline int tile_slots(int t) { return t == kBig || t == kDeep ? 256 : 512; }  // workgroups the chip holds at once

// Microseconds of one step of 128 bytes of k on a chip full of tiles, and on one with a tile per CU.
// Measured on N = 4096, V = 151936, d = 4352 (bf16): 4.08 ms in 256 x 256 tiles, 5.24 in 128 x 128, 6.83
// in 128 x 64; the narrow ones on the shapes above.
inline double step_us(int t, bool full, int es) {
  if (es == 4) return t == kSmall ? (full ? 1.1 : 0.6) : full ? 1.9 : 1.1;
  return t == kBig ? 1.6 : t == kDeep ? 0.45 : t == kSmall ? (full ? 0.55 : 0.36) : t == kMid ? (full ? 1.04 : 0.62) : (full ? 0.68 : 0.4);
}
inline double tiles_us(long long tiles, int t, int steps, int es) {
  const long long slots = tile_slots(t), rounds = tiles / slots, rest = tiles % slots;
  return steps * (rounds * step_us(t, true, es) + (rest > 256 ? step_us(t, true, es) : rest > 0 ? step_us(t, false, es) : 0));
}

// How a product's rows are shared out: the first `head` rows of the longer side in 256 x 256 tiles, the
// others in `tail` tiles (head = 0: one shape for all).  A last round that fills a quarter of the chip
// with 256 x 256 tiles costs as much as a full one: its rows go to smaller tiles instead.
struct Shape {
  bool along_a;     // the rows shared out are A's
  long long head;
  int tail;
};

inline Shape pick_shape(long long rowsA, long long rowsB, int kbytes, int es, bool store = false) {
  const int steps = ceil_div(kbytes, kStepBytes);
  auto cost = [&](long long a, long long b, int t) {
    return a && b ? tiles_us((long long)ceil_div(a, tile_m(t)) * ceil_div(b, tile_n(t)), t, steps, es) : 0.0;
  };
  if (es == 4) return Shape{rowsA >= rowsB, 0, cost(rowsA, rowsB, kSmall) < cost(rowsA, rowsB, kThin) ? kSmall : kThin};
  Shape best{rowsA >= rowsB, 0, rowsB <= 64 && !store ? kThin : kMid};   // dW has no narrow tiles
  double us = cost(rowsA, rowsB, best.tail);
  if (!store)
    for (int t : {kDeep, kSmall})
      if (cost(rowsA, rowsB, t) < us) {
        best.tail = t;
        us = cost(rowsA, rowsB, t);
      }
  if (cost(rowsA, rowsB, kBig) <= us) {
    best.tail = kBig;
    us = cost(rowsA, rowsB, kBig);
  }
  const long long len = best.along_a ? rowsA : rowsB, other = best.along_a ? rowsB : rowsA;
  const long long across = ceil_div(other, 256);
  const long long rounds = (long long)ceil_div(len, 256) * across / 256;
  const long long head = rounds * 256 / across * 256;   // rows whose tiles fill whole rounds
  if (rounds > 0 && head < len) {
    const double mixed = cost(best.along_a ? head : rowsA, best.along_a ? rowsB : head, kBig) +
                         cost(best.along_a ? len - head : rowsA, best.along_a ? rowsB : len - head, kMid) + 4.0;
    if (mixed < us) {
      best.head = head;
      best.tail = kMid;
    }
  }
  return best;
}

// Strips of kStats over V rows of A.
inline int stat_strips(long long V, long long N, int kbytes, int es) {
  const Shape sh = pick_shape(V, N, kbytes, es);
  const long long head = sh.along_a ? sh.head : 0;
  const int tail = sh.along_a || sh.head == 0 ? sh.tail : kBig;
  return (int)(head / strip_rows(kBig)) + ceil_div(V - head, tile_m(tail)) * (tile_m(tail) / strip_rows(tail));
}

// Every launch's work-items fit the 32-bit grid size of the dispatch packet, whatever the tiles (64 x 64
// ones are taken up to some 7000 of them; the parts of kAcc add at most 16 times the tiles of two rounds).
inline bool head_fits(long long N, long long V, long long d) {
  const long long most = 0xffffffffll - 256ll * 1024 * 32;
  return (long long)ceil_div(V, 128) * ceil_div(N, 64) * 256 <= most && N * round_to(d, 1024) / 2 + 512 <= most &&
         (long long)ceil_div(V, 128) * ceil_div(d, 64) * 256 <= most;
}

inline bool head_ok(int N, int V, int d, int dtype) {
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return false;
  if (N < 1 || N > SPEC_MAX_HEAD_ROWS || V < 1 || V > SPEC_MAX_V || d < 1 || d > SPEC_MAX_HEAD_WIDTH) return false;
  return (d * (dtype == SPEC_BF16 ? 2 : 4)) % 16 == 0;
}

// The backward's pieces and its workspace.
struct BackPlan {
  int es, step;          // element size, elements per 128 bytes
  int pieces, vc;        // vocabulary pieces of vc tokens (a multiple of 256; the last may be shorter)
  long long npad;
  int tile, whole, parts;   // of dH: tiles taken whole, and the workgroups that share each of the others
  size_t gn, gt, wt, ht, acc, acc_parts, glab, first, side;   // bytes
  size_t total() const { return gn + gt + wt + ht + acc + acc_parts + glab + first + side; }
};

constexpr long long kPieceBytes = 128ll << 20;   // of G (fp32: and of G^T and W^T) per piece
constexpr int kMaxParts = 16, kPartSteps = 8;    // workgroups per tile at most; steps of one at least

inline BackPlan back_plan(int N, int V, int d, int dtype) {
  BackPlan p{};
  p.es = dtype == SPEC_BF16 ? 2 : 4;
  p.step = kStepBytes / p.es;
  p.npad = round_to(N, p.step);
  const long long rows = round_to(N, 256);                           // whole tiles of rows
  const long long widest = p.es == 4 && d > rows ? d : rows;         // fp32: W^T of the piece, too
  long long vmax = kPieceBytes / (widest * p.es) / 256 * 256;
  // fewer rows than a tile per CU needs are no piece (fp32, 64 x 32768, d = 4096: four pieces of 140 us for
  // kGradZ, 154 us in one)
  const long long least = round_to(256ll * 128 * 64 / round_to(N, 64), 256);
  if (vmax < least) vmax = least;
  p.pieces = ceil_div(V, vmax);
  p.vc = (int)round_to(ceil_div(V, p.pieces), 256);
  p.pieces = ceil_div(V, p.vc);
  // dH has few tiles and a long contraction: whole rounds of tiles are taken a workgroup each, and each
  // tile of the last, partial round is shared by `parts` workgroups along the contraction (272 tiles of
  // 256 x 256 on 256 CUs: one round and 16 tiles by 16 workgroups, 1.06 rounds in place of 2)
  const int steps = p.vc / p.step;
  double best = 1e300;
  const int wide = p.es == 4 || N <= 64 ? kThin : kBig, narrow = p.es == 4 ? kSmall : N <= 64 ? kThin : kMid;
  for (int t : {wide, narrow}) {
    const long long tiles = (long long)ceil_div(d, tile_m(t)) * ceil_div(N, tile_n(t));
    const long long whole = tiles / tile_slots(t) * tile_slots(t), rest = tiles - whole;
    for (int parts = 1; parts <= kMaxParts && (parts == 1 || steps / parts >= kPartSteps); ++parts) {
      // a part costs its share of the steps, and about 6 steps to start and to store
      const double us = tiles_us(whole, t, steps + 6, p.es) + tiles_us(rest * parts, t, ceil_div(steps, parts) + 6, p.es);
      if (us < best) {
        best = us;
        p.tile = t;
        p.whole = (int)whole;
        p.parts = parts;
        p.acc_parts = round_bytes((size_t)rest * (parts - 1) * tile_m(t) * tile_n(t) * sizeof(float));
      }
    }
  }
  p.gn = round_bytes((size_t)rows * p.vc * p.es);
  if (p.es == 4) {   // transposed copies; bf16 operands are turned as they leave LDS
    p.gt = round_bytes((size_t)p.vc * p.npad * p.es);
    p.wt = round_bytes((size_t)d * p.vc * p.es);
  }
  p.ht = round_bytes((size_t)d * p.npad * p.es);
  p.acc = round_bytes((size_t)N * d * sizeof(float));
  if (p.es == 2) {
    p.glab = round_bytes((size_t)N * sizeof(float));
    p.first = round_bytes((size_t)V * sizeof(int32_t));
    p.side = round_bytes((size_t)N * d * sizeof(float));
  }
  return p;
}

}  // namespace spec
