// Which kernel an adjustment of logits takes, and in how many workgroups (host arithmetic only, also compiled by itself
// in the tests).
#pragma once

#include "xent_plan.hpp"

namespace spec {

constexpr int kSlice = 4096, kLongHistory = 8192;
constexpr int kSlotBits = 12, kSlots = 1 << kSlotBits, kFewThreads = 512, kFewGroups = 512, kMaxBits = 4;

// 16 bytes of a row per thread.
constexpr int slice_threads(bool bf16) { return bf16 ? 512 : 1024; }

struct AdjustPlan {
  int bits;            // the listed tokens alone, in 2^bits classes; -1: slices of the vocabulary
  int slice, threads;
  long long workgroups(long long B, int V) const { return bits >= 0 ? B << bits : B * ceil_div(V, slice); }
};

// A launch's work-items are counted in 32 bits.
constexpr long long kMostItems = 0xffffffffll;

// 2^bits classes: as many as give kFewGroups workgroups while each still has some 256 pairs, and no more tokens to a
// class than fill its table to two thirds (as far as a launch's work-items can be counted).  256 single tokens of
// 151936 after 4096: 256 and 512 workgroups 17.7 us, 1024 21.6, 2048 31; 64 blocks of 17 rows: 256 workgroups 23.9,
// 512 and more 22.
inline int few_bits(int B, int R, long long named) {
  int bits = 0;
  while (bits < kMaxBits && (2ll * B << bits) <= kFewGroups && named * R >= 512ll << bits) ++bits;
  while (bits < kMaxBits && 3 * named > 2ll * kSlots << bits && (2ll * B * kFewThreads << bits) <= kMostItems) ++bits;
  return bits;
}

// Slices of 4096 tokens, 16 bytes of a row per thread: two workgroups a CU or more (64 blocks of 17 rows of 151936
// bf16, half of them live, out of place: 83 us; slices of 2048 91; fp32, half as many blocks: by 512 threads 81, by
// 1024 77).  Every slice's workgroup reads the whole history, and from some 8000 tokens on half as many slices are
// faster (96 x 8 rows of 129280 after 30011 tokens: 115 -> 103 us; after 1000: 70 -> 71).  Not so with biases, whose
// table leaves room for one such workgroup a CU (the same rows with 64 biases a request after 12000 and 30011 tokens: 125
// -> 130 and 174 -> 181; under masks 128 -> 138 and 179 -> 191), nor in fp32, with twice the bytes of a row (48 x 8: 77 ->
// 81 and 90 -> 94; under masks 76 -> 85 and 92 -> 103).
// In place without a mask a row's slice through LDS is only ahead where much of the vocabulary is listed: 64 blocks of
// 17 rows as above, histories of a 32nd of the vocabulary 70 us, of a 16th 81, of an 8th 98; the listed tokens where
// they lie 38, 81 and 141.  256 single tokens likewise: 71, 80 and 106; 21, 36 and 77.
// What the host knows is the histories' room H and the number of biases of all requests: short histories in a wide
// array are taken for long ones (256 single tokens after 500: 13 us with H = 500, 15 with 16384, 51 with 32768; 64 blocks
// of 17 rows: 17 and, from 9481 on, 72), and one request's long list for everybody's short one (100000 biases for one of
// 256 single tokens: its classes do not fit their tables, 3.4 ms in place, 84 us out of place).
inline AdjustPlan plan_adjust(bool bf16, bool copy, bool bias, bool mask, int B, int R, int V, int H, int gamma,
                              int bias_count) {
  const long long named = (long long)H + gamma + bias_count / B;   // tokens of a request at most, or so
  if (!copy && !mask && named <= V / (R == 1 ? 8 : 16)) return {few_bits(B, R, named), 0, kFewThreads};
  if (bf16 && !bias && H > kLongHistory) return {-1, 2 * kSlice, 1024};
  return {-1, kSlice, slice_threads(bf16)};
}

}  // namespace spec
