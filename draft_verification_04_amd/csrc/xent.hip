// Softmax cross entropy of a vocabulary head on gfx950, with its gradients, without stored logits.
//
//   z = H W^T (H [N, d], W [V, d]);  loss_n = ln sum_v exp(z_nv) - z_n,label
//   G = (softmax(z) - onehot(label)) * grad_loss;  dH = G W;  dW = G^T H
//
// Every product runs in one matrix kernel over operands whose rows lie along the contraction
// (out[j][i] = sum_k A[i][k] B[j][k], both row-major with k contiguous), with an epilogue per use:
//   kStats  A = W, B = H: per row and per strip of the vocabulary, the largest logit and the sum of
//           exp against it, and the label's logit; xent_combine_kernel adds the strips in fp64, scaled by
//           fp32 exponentials (an ulp each, three at most on a strip's way; fp64 ones: 9.6 us in place of 7.9).
//   kGradZ  the same product again for a piece of the vocabulary; the epilogue forms G.
//   kAcc    dH += G W over the piece: A = W^T, B = G; fp32 in memory.
//   kStore  dW of the piece: A = H^T, B = G^T; rounded to the storage type.
// W^T, H^T and G^T are read as they lie, turned by the transposing LDS read, in bf16; fp32 takes transposed
// copies (bf16 by copies: 18.1 ms in place of 17.4 on the case below).
// G is rounded to bf16 for its products; the label's entry, as large as the rest of its row together, is corrected
// in fp32.  (An entry as large, of another token that the row is sure of, stays rounded: half a step of bf16,
// as much as the rounding of the result.)
// The pieces bound the memory: G of one piece at a time instead of N V logits.
//
// Bound by the matrix units.  MI355X, N = 4096, V = 151936, d = 4352, bf16 (a product is 5.42 TFLOP): kStats
// 3.98 ms (1360 TFLOP/s), kGradZ in 10 pieces 4.51 ms (1200), kAcc 4.19 ms (1290), kStore 4.28 ms (1270).
//
// Operands in LDS: a step of 128 bytes of k (64 bf16 or 32 fp32) per row, rows 128 bytes apart, the
// 16-byte chunk c of row r stored at c ^ (r & 7), so that the 16 rows an MFMA operand read touches
// fall into different banks.  The chunks go from memory to LDS directly (16 bytes per lane; a wave's
// destination is contiguous, so the swizzle is applied to the source address).  MFMA 16x16x32 bf16,
// or four 16x16x4 fp32 on the same 16-byte fragments (which pairs k differently on both sides alike).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <utility>

#include "common.hpp"
#include "rowseg.hpp"
#include "spec_verify.h"
#include "xent_plan.hpp"

namespace spec {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef unsigned int v2u32 __attribute__((ext_vector_type(2)));

#define SPEC_GLOBAL __attribute__((address_space(1)))
#define SPEC_LDS __attribute__((address_space(3)))

constexpr float kLog2eF = 1.44269504f;
constexpr int kNoRow = INT32_MAX;
constexpr int kFoldSteps = 8;     // fp32: steps summed in one accumulator

enum { kStats = 0, kGradZ = 1, kAcc = 2, kStore = 3 };

struct GemmArgs {
  const char* A;     // [rowsA] rows lda bytes apart
  const char* B;     // [rowsB] rows ldb bytes apart
  size_t lda, ldb;
  int rowsA, rowsB;
  int kbytes;        // of a row (a multiple of 16); the contraction's length times the element size
  int arows;         // rows of a k-major A that exist (past them the last one is read: B is zero there)
  int ti, tj;        // tiles
  int whole, parts;  // tiles taken by one workgroup each; the rest by `parts` workgroups each (kAcc)
  // kStats, kGradZ
  const int32_t* labels;
  int v0;            // vocabulary index of A's first row
  float2* part;      // [strips, rowsB] (largest logit, sum of exp against it), from A's first strip
  float* zlab;       // [rowsB]
  const float* lse;
  const float* grad_loss;
  int V;
  char* gn;          // [rowsB, ldgn bytes]
  char* gt;          // [rowsA, ldgt bytes]
  size_t ldgn, ldgt;
  int vpad, npad;    // columns of gn and gt that are written (zeros past the valid ones)
  // bf16: the labels' entries of G (see finish_label)
  float* glab;       // [N] what the rounding of row n's left out
  int32_t* first;    // [V] the first row with the token as its label (kNoRow: none)
  float* side;       // [N, side_ld] dW of a label's token, unrounded, at its first row
  int side_ld;
  // kAcc, kStore
  float* acc;        // [rowsB, rowsA]: whole tiles and the first part of the others
  float* acc_parts;  // [rest tiles, parts - 1, tile]: their further parts
  int accumulate;
  char* out;         // [rowsB, ldo bytes]
  size_t ldo;
};

template <int ES>
__device__ __forceinline__ f32x4 mma(const v4u32& a, const v4u32& b, f32x4 c) {
  if constexpr (ES == 2) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0,
                                                   0, 0);
  } else {
    const f32x4 x = __builtin_bit_cast(f32x4, a), y = __builtin_bit_cast(f32x4, b);
#pragma unroll
    for (int q = 0; q < 4; ++q) c = __builtin_amdgcn_mfma_f32_16x16x4f32(x[q], y[q], c, 0, 0, 0);
    return c;
  }
}

// Waits until at most N of the wave's loads are in flight and its LDS accesses are done, then the
// workgroup barrier.
template <int N>
__device__ __forceinline__ void wait_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// Scheduling of a half step: R LDS reads spread over its M matrix instructions.
template <int R, int M>
__device__ __forceinline__ void interleave() {
#pragma unroll
  for (int i = 0; i < R; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, M / R > 0 ? M / R : 1, 0);   // matrix instructions
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);                       // then an LDS read
  }
  __builtin_amdgcn_sched_group_barrier(0x008, M % R, 0);
}

// bf16 operands that lie the other way round in memory, k along the rows ("k-major": dH = G W takes W, dW =
// G^T H takes both): the tile keeps the memory's layout, 64 rows of k and W columns, and the transposing
// LDS read (ds_read_b64_tr_b16: 16 lanes bring 4 rows of 16 values, lane i takes column i) turns it.  Its
// 16 lanes touch 4 rows of k, 32 bytes each, and a wave rows 8 apart as well: the 32-byte segment s of row
// r is stored at s ^ kswz(r), so that they fall into different banks.
__device__ __forceinline__ int kswz(int row) { return (row & 3) | ((row >> 1) & 4); }

__device__ __forceinline__ v2u32 read_tr(const SPEC_LDS char* p) {
  typedef short s16x4 __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(v2u32, __builtin_amdgcn_ds_read_tr16_b64_v4i16((SPEC_LDS s16x4*)p));
}

// A row takes part in the gradient: a label in range and a finite normaliser.
__device__ __forceinline__ bool live_row(int label, float lse, int V) {
  return label >= 0 && label < V && fabsf(lse) < INFINITY;
}

// Tile of block `bid` of `total`: blocks go round the 8 XCDs, so each XCD takes a contiguous run of
// tiles, ordered in bands of up to 8 j tiles (an XCD's 32 CUs share 4 + 8 operand strips in its L2).
__device__ __forceinline__ int xcd_tile(int bid, int total) {
  const int x = bid & 7, i = bid >> 3, q = total >> 3, rem = total & 7;
  return x < rem ? x * (q + 1) + i : rem * (q + 1) + (x - rem) * q + i;
}

template <int ES, int BM, int BN, int WM, int WN, int ST, int KIND>
__global__ __launch_bounds__(WM * WN * 64) void xent_gemm_kernel(GemmArgs g) {
  constexpr int NTHR = WM * WN * 64, NW = WM * WN;
  constexpr int MT = BM / WM / 16, NT = BN / WN / 16;
  constexpr int CA = BM * 8 / NTHR, CB = BN * 8 / NTHR;   // 16-byte chunks per thread and step
  constexpr int STAGE = (BM + BN) * kStepBytes;
  __shared__ __attribute__((aligned(128))) char lds_[ST * STAGE];
  SPEC_LDS char* const lds = (SPEC_LDS char*)lds_;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wi = wave % WM, wj = wave / WM;
  const int l16 = lane & 15, q = lane >> 4;

  int tile, part = 0, steps = (g.kbytes + kStepBytes - 1) / kStepBytes, step0 = 0;
  if ((int)blockIdx.x < g.whole) {
    tile = xcd_tile((int)blockIdx.x, g.whole);
  } else {
    const int u = (int)blockIdx.x - g.whole;
    tile = g.whole + u / g.parts;
    part = u % g.parts;
    step0 = (int)((long long)steps * part / g.parts);
    steps = (int)((long long)steps * (part + 1) / g.parts);
  }
  const int band = tile / (8 * g.ti), in = tile - band * 8 * g.ti;
  const int bw = min(8, g.tj - band * 8);
  const int i0 = in / bw * BM, j0 = (band * 8 + in % bw) * BN;

  constexpr bool AK = ES == 2 && (KIND == kAcc || KIND == kStore), BK = ES == 2 && KIND == kStore;   // k-major
  constexpr int KROWS = kStepBytes / ES;   // of k per step
  const int kb = step0 * kStepBytes, kbytes = min(steps * kStepBytes, g.kbytes) - kb;
  const int krows = AK ? min(kbytes / ES, g.arows - step0 * KROWS) : 0;
  const int full = AK ? krows / KROWS : kbytes / kStepBytes, rem = kbytes % kStepBytes;
  const int nk = (kbytes + kStepBytes - 1) / kStepBytes;
  const char* A = g.A + (AK ? (size_t)step0 * KROWS * g.lda + (size_t)i0 * ES : (size_t)i0 * g.lda + kb);
  const char* B = g.B + (BK ? (size_t)step0 * KROWS * g.ldb + (size_t)j0 * ES : (size_t)j0 * g.ldb + kb);
  const size_t stepA = AK ? (size_t)KROWS * g.lda : kStepBytes, stepB = BK ? (size_t)KROWS * g.ldb : kStepBytes;

  // Chunk u of this thread.  Rows along k: row (u NW + wave) 8 + lane / 8 of the operand (clamped to the last
  // one), stored at chunk lane % 8 and so read from chunk (lane % 8) ^ (row % 8).  k-major: row (u NW + wave)
  // 64 / L + lane / L of the step, L = lanes per row, 32-byte segment swizzled by the row (columns clamped
  // to the last chunk of the row).
  const int lr = lane >> 3, lc = ((lane & 7) ^ lr) * 16;
  // (k-major: the chunks of a thread lie 16 rows apart, which the swizzle does not see: one lane offset)
  constexpr int LA = BM * ES / 16, LB = BN * ES / 16;
  static_assert(!AK || (NW * (64 / LA) == 16 && LA >= 16), "k-major chunks 16 rows apart");
  static_assert(!BK || (NW * (64 / LB) == 16 && LB >= 16), "k-major chunks 16 rows apart");
  constexpr bool B1 = BK || (AK && KIND == kAcc);   // one lane offset for B, too: dH's B has rows for whole tiles
  uint32_t va[AK ? 1 : CA], vb[B1 ? 1 : CB];
  if constexpr (AK) {
    const int r = wave * (64 / LA) + lane / LA;
    va[0] = (uint32_t)r * (uint32_t)g.lda + min(((lane % LA) ^ (kswz(r) << 1)) * 16, (g.rowsA - i0) * ES - 16);
  } else {
#pragma unroll
    for (int u = 0; u < CA; ++u) va[u] = (uint32_t)min((u * NW + wave) * 8 + lr, g.rowsA - 1 - i0) * (uint32_t)g.lda + lc;
  }
  if constexpr (BK) {   // whole tiles of columns are allocated
    const int r = wave * (64 / LB) + lane / LB;
    vb[0] = (uint32_t)r * (uint32_t)g.ldb + ((lane % LB) ^ (kswz(r) << 1)) * 16;
  } else if constexpr (B1) {
    vb[0] = (uint32_t)(wave * 8 + lr) * (uint32_t)g.ldb + lc;
  } else {
#pragma unroll
    for (int u = 0; u < CB; ++u) vb[u] = (uint32_t)min((u * NW + wave) * 8 + lr, g.rowsB - 1 - j0) * (uint32_t)g.ldb + lc;
  }

  // a thin tile's rows of A are in no other tile: nontemporal (64 rows, V = 129280, d = 4096: 178 -> 163 us)
  constexpr bool ONCE = ES == 2 && BN == 64 && ST == 3;
  auto dma_a = [&](const char* src, uint32_t off, SPEC_LDS char* dst) {
    __builtin_amdgcn_global_load_lds((const SPEC_GLOBAL void*)(src + off), (SPEC_LDS void*)dst, 16, 0, ONCE ? 2 : 0);
  };
  auto dma_b = [&](const char* src, uint32_t off, SPEC_LDS char* dst) {
    __builtin_amdgcn_global_load_lds((const SPEC_GLOBAL void*)(src + off), (SPEC_LDS void*)dst, 16, 0, 0);
  };
  auto issue_whole = [&](SPEC_LDS char* dst, int t) {   // a step of 128 bytes
    dst += wave * 1024;
    // scalar base + 32-bit lane offset (the compiler would otherwise keep 64-bit lane pointers in registers)
    size_t oa = t * stepA, ob = t * stepB;
    asm("" : "+s"(oa), "+s"(ob));
    const char* a = A + oa;
    const char* b = B + ob;
#pragma unroll
    for (int u = 0; u < CA; ++u) dma_a(AK ? a + u * 16 * g.lda : a, va[AK ? 0 : u], dst + u * NW * 1024);
#pragma unroll
    for (int u = 0; u < CB; ++u)
      dma_b(B1 ? b + u * (BK ? 16 : NW * 8) * g.ldb : b, vb[B1 ? 0 : u], dst + BM * kStepBytes + u * NW * 1024);
  };
  // The last step of rows that are no multiple of 128 bytes: zeros behind their end.  Of a k-major A whose
  // rows end within the step: the last row again.
  auto issue_rest = [&](SPEC_LDS char* dst, int t) {
    dst += wave * 1024;
    const char* a = A + t * stepA;
    const char* b = B + t * stepB;
    if constexpr (AK) {
      const int last = krows - 1 - t * KROWS;
#pragma unroll
      for (int u = 0; u < CA; ++u) {
        const int past = max((u * NW + wave) * (64 / LA) + lane / LA - last, 0);
        dma_a(a + u * 16 * g.lda - (size_t)past * g.lda, va[0], dst + u * NW * 1024);
      }
#pragma unroll
      for (int u = 0; u < CB; ++u)
        dma_b(B1 ? b + u * (BK ? 16 : NW * 8) * g.ldb : b, vb[B1 ? 0 : u], dst + BM * kStepBytes + u * NW * 1024);
    } else {
      const v4u32 zero = {};
      dst += lane * 16;
#pragma unroll
      for (int u = 0; u < CA; ++u)
        *reinterpret_cast<SPEC_LDS v4u32*>(dst + u * NW * 1024) = lc < rem ? *reinterpret_cast<const v4u32*>(a + va[AK ? 0 : u]) : zero;
#pragma unroll
      for (int u = 0; u < CB; ++u)
        *reinterpret_cast<SPEC_LDS v4u32*>(dst + BM * kStepBytes + u * NW * 1024) =
            lc < rem ? *reinterpret_cast<const v4u32*>(b + vb[B1 ? 0 : u]) : zero;
    }
  };
  auto issue = [&](int t) {
    if (t < full) issue_whole(lds + (t % ST) * STAGE, t);
    else if (t < nk) issue_rest(lds + (t % ST) * STAGE, t);
  };

  f32x4 c[MT][NT] = {};
  const int ra = (wi * MT * 16 + l16) * kStepBytes, rb = BM * kStepBytes + (wj * NT * 16 + l16) * kStepBytes;
  // k-major: the lane's row of k within a group of four, its 8 bytes of the 32, its segment against the swizzle
  const int kr = l16 >> 2, k8 = (l16 & 3) * 8, sz = kr | ((q & 1) << 2);
  const int ta = (q * 8 + kr) * BM * ES + k8 + ((wi * MT) ^ sz) * 32;
  const int tb = BM * kStepBytes + (q * 8 + kr) * BN * ES + k8 + ((wj * NT) ^ sz) * 32;
  struct Frag {
    v4u32 a[MT], b[NT];
  };
  auto fetch = [&](Frag& f, const SPEC_LDS char* base, int kk) {   // half kk of a step
    const SPEC_LDS char* src = base + ((kk * 4 + q) ^ (lane & 7)) * 16;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      if constexpr (AK) {
        const SPEC_LDS char* p = base + ((ta ^ (m * 32)) + kk * 32 * BM * ES);
        const v2u32 x = read_tr(p), y = read_tr(p + 4 * BM * ES);
        f.a[m] = v4u32{x.x, x.y, y.x, y.y};
      } else {
        f.a[m] = *reinterpret_cast<const SPEC_LDS v4u32*>(src + ra + m * 16 * kStepBytes);
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      if constexpr (BK) {
        const SPEC_LDS char* p = base + ((tb ^ (n * 32)) + kk * 32 * BN * ES);
        const v2u32 x = read_tr(p), y = read_tr(p + 4 * BN * ES);
        f.b[n] = v4u32{x.x, x.y, y.x, y.y};
      } else {
        f.b[n] = *reinterpret_cast<const SPEC_LDS v4u32*>(src + rb + n * 16 * kStepBytes);
      }
    }
  };
  constexpr int READS = MT * (AK ? 2 : 1) + NT * (BK ? 2 : 1);
  auto multiply = [&](const Frag& f) {
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) c[m][n] = mma<ES>(f.a[m], f.b[n], c[m][n]);
  };
  // Half a step ahead: while one half step's operands are multiplied the next one's are read from LDS (22.4
  // -> 18.3 ms on the case above against reading them behind the barrier).  A
  // turn starts behind the barrier: every wave has read all of step t (its second half, f1, is still to be
  // multiplied), whose buffer takes step t + ST, and step t + 1 has landed.  The buffers are restrict
  // arguments: the compiler would otherwise have every read wait for the loads in flight.
  constexpr int MM = MT * NT * (ES == 2 ? 1 : 4);
  Frag f0, f1;
  // fp32: the sums of kFoldSteps steps (256 of k) go to a second accumulator, so that a product is rounded 256 +
  // k / 256 times and not k: errors a third to a fifth (64 x 8000, d = 2048: loss 1.4e-5 -> 3.3e-6, gradients
  // 1.5e-6 -> 0.4e-6 relative; a library's product: as without) for 1 to 3 % of the time (119.6 -> 124.3 us;
  // 128 of k: 0.3e-6 for 1 % more).  bf16: the operands' own rounding is 2^15 times as large.
  constexpr bool FOLD = ES == 4;
  f32x4 folded[MT][NT] = {};
  auto fold = [&](int t) {   // behind turn t, which ends with the first half of step t + 1
    if (!FOLD || t % kFoldSteps != kFoldSteps - 2) return;
#pragma unroll
    for (int m = 0; m < MT; ++m)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        folded[m][n] += c[m][n];
        c[m][n] = f32x4{};
      }
  };
  auto turn = [&](SPEC_LDS char* __restrict__ free, const SPEC_LDS char* __restrict__ cur, int t) {
    issue_whole(free, t + ST);
    fetch(f0, cur, 0);
    multiply(f1);
    __builtin_amdgcn_sched_group_barrier(0x010, CA + CB, 0);   // the loads from memory first (last: kStats + 14%)
    interleave<READS, MM>();
    fetch(f1, cur, 1);
    multiply(f0);
    interleave<READS, MM>();
  };
#pragma unroll
  for (int t = 0; t < ST; ++t) issue(t);
  if (nk > 0) {
    if (nk >= ST) wait_barrier<(ST - 1) * (CA + CB)>();
    else wait_barrier<0>();
    fetch(f0, lds, 0);
    fetch(f1, lds, 1);
    multiply(f0);
    if (nk >= ST) wait_barrier<(ST - 2) * (CA + CB)>();
    else wait_barrier<0>();
    int t = 0;
    for (; t + ST < full; ++t) {
      turn(lds + (t % ST) * STAGE, lds + ((t + 1) % ST) * STAGE, t);
      fold(t);
      wait_barrier<(ST - 2) * (CA + CB)>();
    }
    for (; t + 1 < nk; ++t) {
      issue(t + ST);
      fetch(f0, lds + ((t + 1) % ST) * STAGE, 0);
      multiply(f1);
      fetch(f1, lds + ((t + 1) % ST) * STAGE, 1);
      multiply(f0);
      fold(t);
      wait_barrier<0>();
    }
    multiply(f1);
    if constexpr (FOLD) {
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) c[m][n] += folded[m][n];
    }
  }

  // c[m][n][x]: row i = iw + 16 m + x of A (consecutive in x), row j of B = jw + 16 n
  const int iw = i0 + wi * MT * 16 + q * 4, jw = j0 + wj * NT * 16 + l16;
  if constexpr (KIND == kStats) {
    const bool edge = i0 + BM > g.rowsA;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int j = jw + n * 16;
      float mx = -INFINITY;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if (edge && iw + m * 16 + x >= g.rowsA) c[m][n][x] = -INFINITY;
          mx = fmaxf(mx, c[m][n][x]);
        }
      mx = fmaxf(mx, __shfl_xor(mx, 16));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      const float ref = mx > -INFINITY ? mx : 0.f;
      float s = 0.f;
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int x = 0; x < 4; ++x) s += __builtin_amdgcn_exp2f((c[m][n][x] - ref) * kLog2eF);
      s += __shfl_xor(s, 16);
      s += __shfl_xor(s, 32);
      if (j < g.rowsB) {
        if (q == 0) g.part[(size_t)(i0 / (BM / WM) + wi) * g.rowsB + j] = make_float2(mx, s);
        const int rel = g.labels[j] - g.v0 - iw;   // the lane that holds the label's logit writes it
        if (rel >= 0 && rel < MT * 16 && (rel & 15) < 4 && iw + rel < g.rowsA) {
          float z = 0.f;
#pragma unroll
          for (int m = 0; m < MT; ++m)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (rel == m * 16 + x) z = c[m][n][x];
          g.zlab[j] = z;
        }
      }
    }
  } else if constexpr (KIND == kGradZ) {
    const bool edge = i0 + BM > g.rowsA;
    int labels[NT];
    float lses[NT], scales[NT];
#pragma unroll
    for (int n = 0; n < NT; ++n) {   // ahead of the stores, which would hold them up
      const int jc = min(jw + n * 16, g.rowsB - 1);
      labels[n] = g.labels[jc];
      lses[n] = g.lse[jc];
      scales[n] = g.grad_loss[jc];
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int j = jw + n * 16;
      const int label = labels[n];
      const float lse = lses[n], s = scales[n];
      const bool live = j < g.rowsB && live_row(label, lse, g.V);
      auto prob = [&](float z) { return __builtin_amdgcn_exp2f((z - lse) * kLog2eF); };
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int i = iw + m * 16;
        f32x4 o;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          o[x] = live ? prob(c[m][n][x]) * s : 0.f;
          if (edge && i + x >= g.rowsA) o[x] = 0.f;
        }
        if constexpr (ES == 2) {
          bf16x4 h;
#pragma unroll
          for (int x = 0; x < 4; ++x) h[x] = (__bf16)o[x];
          if (j < g.npad && i < g.vpad) *reinterpret_cast<bf16x4*>(g.gn + (size_t)j * g.ldgn + (size_t)i * 2) = h;
        } else {
          if (j < g.rowsB && i < g.vpad) *reinterpret_cast<f32x4*>(g.gn + (size_t)j * g.ldgn + (size_t)i * 4) = o;
          if (j < g.npad)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (i + x < g.rowsA) *reinterpret_cast<float*>(g.gt + (size_t)(i + x) * g.ldgt + (size_t)j * 4) = o[x];
        }
      }
      // the label's entry over it, by the lane that holds its logit (out of the loop above: kGradZ of the case
      // above 469 -> 451 us a piece)
      const int lab = label - g.v0, rel = lab - iw;
      if (live && rel >= 0 && rel < MT * 16 && (rel & 15) < 4 && lab < g.rowsA) {
        float z = 0.f;
#pragma unroll
        for (int m = 0; m < MT; ++m)
#pragma unroll
          for (int x = 0; x < 4; ++x)
            if (rel == m * 16 + x) z = c[m][n][x];
        const float o = (prob(z) - 1.f) * s;
        if constexpr (ES == 2) {
          const __bf16 h = (__bf16)o;
          *reinterpret_cast<__bf16*>(g.gn + (size_t)j * g.ldgn + (size_t)lab * 2) = h;
          g.glab[j] = o - (float)h;
          if (g.first) atomicMin(&g.first[label], j);
        } else {
          *reinterpret_cast<float*>(g.gn + (size_t)j * g.ldgn + (size_t)lab * 4) = o;
          *reinterpret_cast<float*>(g.gt + (size_t)lab * g.ldgt + (size_t)j * 4) = o;
        }
      }
    }
  } else {
    int firsts[NT];
    if constexpr (KIND == kStore && ES == 2) {
#pragma unroll
      for (int n = 0; n < NT; ++n) firsts[n] = g.first[g.v0 + min(jw + n * 16, g.rowsB - 1)];
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int j = jw + n * 16;
      if (j >= g.rowsB) continue;
      int first = kNoRow;
      if constexpr (KIND == kStore && ES == 2) first = firsts[n];
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int i = iw + m * 16;
        if (i >= g.rowsA) continue;   // rowsA is a multiple of 4
        f32x4 o = c[m][n];
        if constexpr (KIND == kAcc) {
          f32x4* p = reinterpret_cast<f32x4*>(
              part == 0 ? g.acc + (size_t)j * g.rowsA + i
                        : g.acc_parts + ((size_t)((tile - g.whole) * (g.parts - 1) + part - 1) * BN + (j - j0)) * BM +
                              (i - i0));
          if (g.accumulate) o += *p;
          *p = o;
        } else if constexpr (ES == 2) {
          bf16x4 h;
#pragma unroll
          for (int x = 0; x < 4; ++x) h[x] = (__bf16)o[x];
          if (first != kNoRow) *reinterpret_cast<f32x4*>(g.side + (size_t)first * g.side_ld + i) = o;
          else *reinterpret_cast<bf16x4*>(g.out + (size_t)j * g.ldo + (size_t)i * 2) = h;
        } else {
          *reinterpret_cast<f32x4*>(g.out + (size_t)j * g.ldo + (size_t)i * 4) = o;
        }
      }
    }
  }
}

// Strips -> lse, loss and status per row: R rows per workgroup, 1024 / R threads share a row's strips
// (each a running maximum and fp64 sum; R = 16 reads whole lines, R = 1 spreads few rows over the chip).
constexpr int kCombineThreads = 1024;

template <int R>
__global__ __launch_bounds__(kCombineThreads) void xent_combine_kernel(const float2* part, int strips, int N, int V,
                                                                       const int32_t* labels, const float* zlab,
                                                                       float* loss, float* lse, int32_t* status) {
  constexpr int H = kCombineThreads / R, U = 4;
  __shared__ float sm[R][H + 1];
  __shared__ double ss[R][H + 1];
  const int r = threadIdx.x % R, h = threadIdx.x / R;
  const int n = (int)blockIdx.x * R + r, nc = min(n, N - 1);
  float m = -INFINITY;
  double s = 0.0;
  for (int t = h; t < strips; t += U * H) {
    float2 p[U];
#pragma unroll
    for (int u = 0; u < U; ++u) p[u] = part[(size_t)min(t + u * H, strips - 1) * N + nc];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (t + u * H >= strips) break;
      const float M = fmaxf(m, p[u].x), d = M > -INFINITY ? M : 0.f;
      s = s * (double)__builtin_amdgcn_exp2f((m - d) * kLog2eF) +
          (double)p[u].y * (double)__builtin_amdgcn_exp2f((p[u].x > -INFINITY ? p[u].x - d : 0.f) * kLog2eF);
      m = M;
    }
  }
  sm[r][h] = m;
  ss[r][h] = s;
  __syncthreads();
  // a wave per row joins its H values
  const int wave = (int)threadIdx.x >> 6, lane = (int)threadIdx.x & 63;
  if (wave >= R || (int)blockIdx.x * R + wave >= N) return;
  const int row = (int)blockIdx.x * R + wave;
  float M = -INFINITY;
  for (int t = lane; t < H; t += SPEC_WAVE) M = fmaxf(M, sm[wave][t]);
  M = wave_max(M);
  double S = 0.0;
  for (int t = lane; t < H; t += SPEC_WAVE)
    S += sm[wave][t] > -INFINITY ? ss[wave][t] * (double)__builtin_amdgcn_exp2f((sm[wave][t] - M) * kLog2eF) : ss[wave][t];
  S = wave_sum(S);
  if (lane == 0) {
    const bool fin = M < INFINITY && M > -INFINITY && S > 0.0 && S < INFINITY;   // NaN sums fail too
    const double ls = log(S);
    const int label = labels[row];
    int st = 0;
    if (label < -1 || label >= V) st |= SPEC_REQ_BAD_TOKEN;
    if (label != -1 && !fin) st |= SPEC_REQ_NONFINITE;
    lse[row] = fin ? (float)((double)M + ls) : NAN;
    loss[row] = label == -1 ? 0.f : (st ? NAN : (float)((double)M - (double)zlab[row] + ls));
    if (status) status[row] = st;
  }
}

// fp32: out[c][r] = in[r][c], r < R valid and not left out (else 0) for r < rpad; 64 x 64 tiles.
__global__ __launch_bounds__(256) void xent_transpose_kernel(const char* in, size_t ldi, int R, int C, char* out,
                                                             size_t ldo, int rpad, const int32_t* labels,
                                                             const float* lse, int V) {
  __shared__ uint32_t t[64][65];
  const int r0 = (int)blockIdx.x * 64, c0 = (int)blockIdx.y * 64, tid = threadIdx.x;
  for (int u = tid; u < 64 * 16; u += 256) {
    const int r = u / 16, c = u % 16 * 4;
    v4u32 v = {};
    const bool on = r0 + r < R && c0 + c < C;
    if (on && (!labels || live_row(labels[r0 + r], lse[r0 + r], V)))
      v = *reinterpret_cast<const v4u32*>(in + (size_t)(r0 + r) * ldi + (size_t)(c0 + c) * 4);
#pragma unroll
    for (int x = 0; x < 4; ++x) t[r][c + x] = v[x];
  }
  __syncthreads();
  for (int u = tid; u < 64 * 16; u += 256) {
    const int c = u / 16, r = u % 16 * 4;
    if (c0 + c < C && r0 + r < rpad)
      *reinterpret_cast<v4u32*>(out + (size_t)(c0 + c) * ldo + (size_t)(r0 + r) * 4) =
          v4u32{t[r][c], t[r + 1][c], t[r + 2][c], t[r + 3][c]};
  }
}

// bf16, before dW: H with zeros in the rows left out (and up to npad rows; 0 * inf would reach dW otherwise),
// and no first rows yet.
__global__ __launch_bounds__(256) void xent_prepare_kernel(const v4u32* in, int N, int d8, v4u32* out, long long n8,
                                                           const int32_t* labels, const float* lse, int V,
                                                           int32_t* first) {
  const long long t = (long long)blockIdx.x * 256 + threadIdx.x;
  if (t < V) first[t] = kNoRow;
  if (t >= n8) return;
  const int r = (int)(t / d8);
  v4u32 v = {};
  if (r < N && live_row(labels[r], lse[r], V)) v = in[t];
  out[t] = v;
}

// grad_hidden = the sums, the parts of a shared tile added in order, rounded once; zeros for the rows
// left out.
template <int ES>
__device__ __forceinline__ void finish_hidden(const GemmArgs& g, int bm, int bn, char* out, const char* weight, size_t t) {
  const int d = g.rowsA, N = g.rowsB, d4 = d / 4;
  if (t >= (size_t)N * d4) return;
  const int n = (int)(t / d4), i = (int)(t - (size_t)n * d4) * 4;
  f32x4 s = {};
  const int label = g.labels[n];
  if (live_row(label, g.lse[n], g.V)) {
    s = reinterpret_cast<const f32x4*>(g.acc)[t];
    const int ti = i / bm, tj = n / bn, band = tj / 8;
    const int rest = band * 8 * g.ti + ti * min(8, g.tj - band * 8) + tj % 8 - g.whole;
    if (rest >= 0)
      for (int p = 0; p < g.parts - 1; ++p)
        s += *reinterpret_cast<const f32x4*>(g.acc_parts + ((size_t)(rest * (g.parts - 1) + p) * bn + (n - tj * bn)) * bm +
                                             (i - ti * bm));
    if constexpr (ES == 2) {   // what the rounding of the label's G left out
      const bf16x4 w = *reinterpret_cast<const bf16x4*>(weight + ((size_t)label * d + i) * 2);
      const float r = g.glab[n];
#pragma unroll
      for (int x = 0; x < 4; ++x) s[x] += r * (float)w[x];
    }
  }
  if constexpr (ES == 2) {
    bf16x4 h;
#pragma unroll
    for (int x = 0; x < 4; ++x) h[x] = (__bf16)s[x];
    reinterpret_cast<bf16x4*>(out)[t] = h;
  } else {
    reinterpret_cast<f32x4*>(out)[t] = s;
  }
}

// dW of the tokens that are labels (bf16): the label's entry of G, (p - 1) grad_loss, is as large as the rest of
// its row together, and its rounding alone would add as much again to the gradient's error.  The product
// leaves these tokens' sums unrounded at their first row; the workgroups of that row (one per 1024 columns)
// add, in row order, what the rounding left out times the hidden state of every row with the label, and
// round once.
constexpr int kLabelThreads = 256;

__device__ __forceinline__ void finish_label(const GemmArgs& g, int n, int part, const char* hidden, char* out) {
  const int32_t* labels = g.labels;
  const float* lse = g.lse;
  const float* glab = g.glab;
  const int32_t* first = g.first;
  const float* side = g.side;
  const int N = g.rowsB, V = g.V, d = g.rowsA;
  constexpr int NW = kLabelThreads / SPEC_WAVE, CHUNK = 4 * kLabelThreads;
  __shared__ int32_t rows[CHUNK];
  __shared__ int cnt[NW];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int label = labels[n];
  if (!live_row(label, lse[n], V) || first[label] != n) return;
  const int d4 = d / 4, c = part * kLabelThreads + tid, cc = min(c, d4 - 1);
  const bf16x4* h4 = reinterpret_cast<const bf16x4*>(hidden) + cc;
  f32x4 s = reinterpret_cast<const f32x4*>(side + (size_t)n * d)[cc];
  for (int m0 = n; m0 < N; m0 += CHUNK) {
    // the rows of the chunk with this label, in order: a wave takes 4 * 64 rows in a row
    unsigned long long hit[4];
    int mine = 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int m = m0 + (wave * 4 + u) * SPEC_WAVE + lane, mc = min(m, N - 1);
      hit[u] = __ballot(m < N && labels[mc] == label && fabsf(lse[mc]) < INFINITY);
      mine += (int)__popcll(hit[u]);
    }
    __syncthreads();   // the last chunk's rows are read
    if (lane == 0) cnt[wave] = mine;
    __syncthreads();
    int base = 0, total = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      base += w < wave ? cnt[w] : 0;
      total += cnt[w];
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      if ((hit[u] >> lane) & 1ull)
        rows[base + (int)__popcll(hit[u] & ((1ull << lane) - 1))] = m0 + (wave * 4 + u) * SPEC_WAVE + lane;
      base += (int)__popcll(hit[u]);
    }
    __syncthreads();
    constexpr int U = 8;   // rows in flight
    for (int e = 0; e < total; e += U) {
      bf16x4 x[U];
      float r[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int m = rows[min(e + u, total - 1)];
        r[u] = glab[m];
        x[u] = h4[(size_t)m * d4];
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (e + u >= total) break;
#pragma unroll
        for (int q = 0; q < 4; ++q) s[q] += r[u] * (float)x[u][q];
      }
    }
  }
  bf16x4 o;
#pragma unroll
  for (int q = 0; q < 4; ++q) o[q] = (__bf16)s[q];
  if (c < d4) reinterpret_cast<bf16x4*>(out + (size_t)label * d * 2)[c] = o;
}

// Both gradients' last step in one launch: `parts` workgroups per row for the labels' tokens of dW, then dH's.
template <int ES>
__global__ __launch_bounds__(kLabelThreads) void xent_finish_kernel(GemmArgs g, int parts, int bm, int bn,
                                                                    const char* hidden, const char* weight,
                                                                    char* grad_hidden, char* grad_weight) {
  const unsigned nl = (unsigned)g.rowsB * (unsigned)parts;
  if (ES == 2 && blockIdx.x < nl)
    finish_label(g, (int)(blockIdx.x / (unsigned)parts), (int)(blockIdx.x % (unsigned)parts), hidden, grad_weight);
  else
    finish_hidden<ES>(g, bm, bn, grad_hidden, weight, (size_t)(blockIdx.x - nl) * kLabelThreads + threadIdx.x);
}

// ---- host -------------------------------------------------------------------

template <int ES, int KIND>
void launch_tiles(GemmArgs& g, int tile, int whole, int parts, hipStream_t s) {
  g.ti = ceil_div(g.rowsA, tile_m(tile));
  g.tj = ceil_div(g.rowsB, tile_n(tile));
  const int tiles = g.ti * g.tj;   // within head_fits
  g.whole = whole < tiles ? whole : tiles;
  g.parts = parts;
  const dim3 grid((unsigned)(g.whole + (tiles - g.whole) * parts));
  const auto go = [&](auto kernel, int threads) { hipLaunchKernelGGL(kernel, grid, dim3(threads), 0, s, g); };
  if constexpr (ES == 4) {
    if (tile == kSmall) go(xent_gemm_kernel<4, 64, 64, 2, 2, 4, KIND>, 256);
    else go(xent_gemm_kernel<4, 128, 64, 2, 2, 3, KIND>, 256);
  } else {
    if (tile == kBig) go(xent_gemm_kernel<2, 256, 256, 2, 4, 2, KIND>, 512);
    else if (tile == kMid) go(xent_gemm_kernel<2, 128, 128, 2, 2, 2, KIND>, 256);
    if constexpr (KIND != kStore) {
      if (tile == kThin) go(xent_gemm_kernel<2, 128, 64, 2, 2, 3, KIND>, 256);
    }
    if constexpr (KIND == kStats || KIND == kGradZ) {
      if (tile == kDeep) go(xent_gemm_kernel<2, 128, 64, 2, 2, 6, KIND>, 256);
      else if (tile == kSmall) go(xent_gemm_kernel<2, 64, 64, 2, 2, 5, KIND>, 256);
    }
  }
}

// A product in the shapes of pick_shape: kStats and kGradZ share out A's rows (the vocabulary), kStore
// the longer side of either.
template <int ES, int KIND>
void launch_gemm(const GemmArgs& g, hipStream_t s) {
  const Shape sh = pick_shape(g.rowsA, g.rowsB, g.kbytes, ES, KIND == kStore);
  const bool split = sh.head > 0 && (sh.along_a || KIND == kStore);
  GemmArgs h = g;
  if (split) {
    GemmArgs f = g;
    (sh.along_a ? f.rowsA : f.rowsB) = (int)sh.head;
    if (KIND == kGradZ) f.vpad = (int)sh.head;
    launch_tiles<ES, KIND>(f, kBig, INT32_MAX, 1, s);
    constexpr bool KM = ES == 2 && KIND == kStore;   // k-major: rows of the product are columns in memory
    if (sh.along_a) {
      h.A += KM ? (size_t)sh.head * ES : (size_t)sh.head * g.lda;
      h.rowsA -= (int)sh.head;
      if (KIND == kStats || KIND == kGradZ) h.v0 += (int)sh.head;
      if (KIND == kStats) h.part += (size_t)(sh.head / strip_rows(kBig)) * g.rowsB;
      if (KIND == kGradZ) {
        h.gn += (size_t)sh.head * ES;
        if (ES == 4) h.gt += (size_t)sh.head * g.ldgt;
        h.vpad -= (int)sh.head;
      }
      if (KIND == kStore) {
        h.out += (size_t)sh.head * ES;
        h.side += sh.head;
      }
    } else {
      h.B += KM ? (size_t)sh.head * ES : (size_t)sh.head * g.ldb;
      h.rowsB -= (int)sh.head;
      h.out += (size_t)sh.head * g.ldo;
      h.v0 += (int)sh.head;
    }
  }
  launch_tiles<ES, KIND>(h, split || sh.head == 0 ? sh.tail : kBig, INT32_MAX, 1, s);
}

template <int ES>
int32_t run_forward(int N, int V, int d, const void* hidden, const void* weight, const int32_t* labels, float* loss,
                    float* lse, int32_t* status, char* ws, hipStream_t s) {
  const int strips = stat_strips(V, N, d * ES, ES);
  GemmArgs g{};
  g.A = reinterpret_cast<const char*>(weight); g.B = reinterpret_cast<const char*>(hidden);
  g.lda = g.ldb = (size_t)d * ES;
  g.rowsA = V; g.rowsB = N; g.kbytes = d * ES;
  g.labels = labels; g.V = V;
  g.part = reinterpret_cast<float2*>(ws);
  g.zlab = reinterpret_cast<float*>(ws + round256((size_t)strips * N * sizeof(float2)));
  launch_gemm<ES, kStats>(g, s);
  if (N >= 2048)
    hipLaunchKernelGGL(xent_combine_kernel<16>, dim3(ceil_div(N, 16)), dim3(kCombineThreads), 0, s, g.part, strips, N,
                       V, labels, g.zlab, loss, lse, status);
  else if (N >= 512)
    hipLaunchKernelGGL(xent_combine_kernel<4>, dim3(ceil_div(N, 4)), dim3(kCombineThreads), 0, s, g.part, strips, N, V,
                       labels, g.zlab, loss, lse, status);
  else
    hipLaunchKernelGGL(xent_combine_kernel<1>, dim3(N), dim3(kCombineThreads), 0, s, g.part, strips, N, V, labels,
                       g.zlab, loss, lse, status);
  return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_ERR_HIP;
}

template <int ES>
int32_t run_backward(int N, int V, int d, int dtype, const void* hidden, const void* weight, const int32_t* labels,
                     const float* lse, const float* grad_loss, void* grad_hidden, void* grad_weight, char* ws,
                     hipStream_t s) {
  const BackPlan p = back_plan(N, V, d, dtype);
  char* gn = ws;
  char* gt = gn + p.gn;
  char* wt = gt + p.gt;
  char* ht = wt + p.wt;
  float* acc = reinterpret_cast<float*>(ht + p.ht);
  GemmArgs h{};   // dH
  h.A = wt; h.lda = (size_t)p.vc * ES; h.rowsA = d;
  h.B = gn; h.ldb = (size_t)p.vc * ES; h.rowsB = N;
  h.acc = acc; h.acc_parts = reinterpret_cast<float*>(ht + p.ht + p.acc);
  h.labels = labels; h.lse = lse; h.V = V;
  char* lab = ht + p.ht + p.acc + p.acc_parts;
  h.glab = reinterpret_cast<float*>(lab);
  int32_t* first = ES == 2 && grad_weight ? reinterpret_cast<int32_t*>(lab + p.glab) : nullptr;
  float* side = reinterpret_cast<float*>(lab + p.glab + p.first);
  const size_t ld = (size_t)d * ES;
  if (grad_weight) {
    if constexpr (ES == 2) {
      const long long n8 = p.npad * (d / 8);
      hipLaunchKernelGGL(xent_prepare_kernel, dim3(ceil_div(n8 > V ? n8 : V, 256)), dim3(256), 0, s,
                         reinterpret_cast<const v4u32*>(hidden), N, d / 8, reinterpret_cast<v4u32*>(ht), n8, labels, lse,
                         V, first);
    } else {
      hipLaunchKernelGGL(xent_transpose_kernel, dim3(ceil_div(p.npad, 64), ceil_div(d, 64)), dim3(256), 0, s,
                         reinterpret_cast<const char*>(hidden), ld, N, d, ht, (size_t)p.npad * ES, (int)p.npad, labels,
                         lse, V);
    }
  }
  for (int c = 0; c < p.pieces; ++c) {
    const int v0 = c * p.vc, nv = V - v0 < p.vc ? V - v0 : p.vc;
    const int vpad = (int)round_to(nv, p.step);
    const char* w = reinterpret_cast<const char*>(weight) + (size_t)v0 * ld;
    GemmArgs g{};
    g.A = w; g.B = reinterpret_cast<const char*>(hidden);
    g.lda = g.ldb = ld;
    g.rowsA = nv; g.rowsB = N; g.kbytes = d * ES;
    g.labels = labels; g.V = V; g.v0 = v0; g.lse = lse; g.grad_loss = grad_loss;
    g.gn = gn; g.ldgn = (size_t)p.vc * ES; g.vpad = vpad;
    g.gt = gt; g.ldgt = (size_t)p.npad * ES; g.npad = (int)p.npad;
    g.glab = h.glab; g.first = first;
    launch_gemm<ES, kGradZ>(g, s);
    if (grad_hidden) {
      if constexpr (ES == 2) {
        h.A = w; h.lda = ld; h.arows = nv;
      } else {
        hipLaunchKernelGGL(xent_transpose_kernel, dim3(ceil_div(vpad, 64), ceil_div(d, 64)), dim3(256), 0, s, w, ld,
                           nv, d, wt, (size_t)p.vc * ES, vpad, nullptr, nullptr, 0);
      }
      h.kbytes = vpad * ES;
      h.accumulate = c > 0;
      launch_tiles<ES, kAcc>(h, p.tile, p.whole, p.parts, s);
    }
    if (grad_weight) {
      GemmArgs w{};
      w.A = ht; w.rowsA = d; w.rowsB = nv;
      if constexpr (ES == 2) {
        w.lda = ld; w.arows = (int)p.npad;
        w.B = gn; w.ldb = (size_t)p.vc * ES;
      } else {
        w.lda = (size_t)p.npad * ES;
        w.B = gt; w.ldb = (size_t)p.npad * ES;
      }
      w.kbytes = (int)p.npad * ES;
      w.out = reinterpret_cast<char*>(grad_weight) + (size_t)v0 * ld; w.ldo = ld;
      w.v0 = v0; w.first = first; w.side = side; w.side_ld = d;
      launch_gemm<ES, kStore>(w, s);
    }
  }
  h.first = first;
  h.side = side;
  const int parts = first ? ceil_div(d, 4 * kLabelThreads) : 0;
  const long long last = (long long)N * parts + (grad_hidden ? ceil_div((long long)N * d / 4, kLabelThreads) : 0);
  if (last)
    hipLaunchKernelGGL(xent_finish_kernel<ES>, dim3((unsigned)last), dim3(kLabelThreads), 0, s, h, parts,
                       tile_m(p.tile), tile_n(p.tile), reinterpret_cast<const char*>(hidden),
                       reinterpret_cast<const char*>(weight), reinterpret_cast<char*>(grad_hidden),
                       reinterpret_cast<char*>(grad_weight));
  return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_ERR_HIP;
}

}  // namespace
}  // namespace spec

using namespace spec;

extern "C" size_t spec_head_xent_workspace_size(int32_t N, int32_t V, int32_t d, int32_t dtype) {
  if (!head_ok(N, V, d, dtype)) return 0;
  const size_t strips = (size_t)stat_strips(V, N, d * (dtype == SPEC_BF16 ? 2 : 4), dtype == SPEC_BF16 ? 2 : 4);
  return round256(strips * N * sizeof(float2)) + round256((size_t)N * sizeof(float));
}

extern "C" int32_t spec_head_xent(int32_t N, int32_t V, int32_t d, int32_t dtype, const void* hidden,
                                  const void* weight, const int32_t* labels, float* loss_out, float* lse_out,
                                  int32_t* status, void* workspace, size_t workspace_bytes, void* stream) {
  if (!head_ok(N, V, d, dtype)) return SPEC_ERR_INVALID_ARG;
  if (!hidden || !weight || !labels || !loss_out || !lse_out) return SPEC_ERR_INVALID_ARG;
  if (!aligned16(hidden) || !aligned16(weight)) return SPEC_ERR_INVALID_ARG;
  if (!workspace || !aligned256(workspace) || workspace_bytes < spec_head_xent_workspace_size(N, V, d, dtype))
    return SPEC_ERR_WORKSPACE;
  if (!head_fits(N, V, d)) return SPEC_ERR_UNSUPPORTED;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  char* ws = reinterpret_cast<char*>(workspace);
  return dtype == SPEC_BF16 ? run_forward<2>(N, V, d, hidden, weight, labels, loss_out, lse_out, status, ws, s)
                            : run_forward<4>(N, V, d, hidden, weight, labels, loss_out, lse_out, status, ws, s);
}

extern "C" size_t spec_head_xent_backward_workspace_size(int32_t N, int32_t V, int32_t d, int32_t dtype) {
  return head_ok(N, V, d, dtype) ? back_plan(N, V, d, dtype).total() : 0;
}

extern "C" int32_t spec_head_xent_backward(int32_t N, int32_t V, int32_t d, int32_t dtype, const void* hidden,
                                           const void* weight, const int32_t* labels, const float* lse,
                                           const float* grad_loss, void* grad_hidden, void* grad_weight,
                                           void* workspace, size_t workspace_bytes, void* stream) {
  if (!head_ok(N, V, d, dtype)) return SPEC_ERR_INVALID_ARG;
  if (!hidden || !weight || !labels || !lse || !grad_loss || (!grad_hidden && !grad_weight))
    return SPEC_ERR_INVALID_ARG;
  if (!aligned16(hidden) || !aligned16(weight) || !aligned16(grad_hidden) || !aligned16(grad_weight))
    return SPEC_ERR_INVALID_ARG;
  if (!workspace || !aligned256(workspace) ||
      workspace_bytes < spec_head_xent_backward_workspace_size(N, V, d, dtype))
    return SPEC_ERR_WORKSPACE;
  // the inputs are read after the first piece's gradients are written
  const size_t row = (size_t)d * (dtype == SPEC_BF16 ? 2 : 4), h_bytes = N * row, w_bytes = V * row;
  for (auto [g, n] : {std::pair<const void*, size_t>{grad_hidden, h_bytes}, {grad_weight, w_bytes}})
    if (overlap(g, n, hidden, h_bytes) || overlap(g, n, weight, w_bytes) || overlap(g, n, labels, N * sizeof(int32_t)) ||
        overlap(g, n, lse, N * sizeof(float)) || overlap(g, n, grad_loss, N * sizeof(float)))
      return SPEC_ERR_INVALID_ARG;
  if (overlap(grad_hidden, h_bytes, grad_weight, w_bytes)) return SPEC_ERR_INVALID_ARG;
  if (!head_fits(N, V, d)) return SPEC_ERR_UNSUPPORTED;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  char* ws = reinterpret_cast<char*>(workspace);
  return dtype == SPEC_BF16
             ? run_backward<2>(N, V, d, dtype, hidden, weight, labels, lse, grad_loss, grad_hidden, grad_weight, ws, s)
             : run_backward<4>(N, V, d, dtype, hidden, weight, labels, lse, grad_loss, grad_hidden, grad_weight, ws, s);
}
