// Softmax cross entropy of a vocabulary head on gfx950, with its gradients, without stored logits.
//
//   z = H W^T (H [N, d], W [V, d]);  loss_n = ln sum_v exp(z_nv) - z_n,label
//   G = (softmax(z) - onehot(label)) * grad_loss;  dH = G W;  dW = G^T H
//
// Every product runs in one matrix kernel over operands whose rows lie along the contraction
// (out[j][i] = sum_k A[i][k] B[j][k], both row-major with k contiguous), with an epilogue per use:
//   kStats  A = W, B = H: per row and per strip of the vocabulary, the largest logit and the sum of
//           exp against it, and the label's logit; xent_combine_kernel adds the strips in fp64.
//   kGradZ  the same product again for a piece of the vocabulary; the epilogue forms G and stores it
//           both ways round, [N, piece] and [piece, N].
//   kAcc    dH += G W over the piece: A = W^T (the piece transposed once), B = G; fp32 in memory.
//   kStore  dW of the piece: A = H^T, B = G^T; rounded to the storage type.
// The pieces bound the memory: G, G^T and W^T of one piece at a time instead of N V logits.
//
// Operands in LDS: a step of 128 bytes of k (64 bf16 or 32 fp32) per row, rows 128 bytes apart, the
// 16-byte chunk c of row r stored at c ^ (r & 7), so that the 16 rows an MFMA operand read touches
// fall into different banks.  The chunks go from memory to LDS directly (16 bytes per lane; a wave's
// destination is contiguous, so the swizzle is applied to the source address).  MFMA 16x16x32 bf16,
// or four 16x16x4 fp32 on the same 16-byte fragments (which pairs k differently on both sides alike).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "common.hpp"
#include "rowseg.hpp"
#include "spec_verify.h"

namespace spec {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

#define SPEC_GLOBAL __attribute__((address_space(1)))
#define SPEC_LDS __attribute__((address_space(3)))

constexpr float kLog2eF = 1.44269504f;
constexpr int kStepBytes = 128;   // of k per row and pipeline step

enum { kStats = 0, kGradZ = 1, kAcc = 2, kStore = 3 };

struct GemmArgs {
  const char* A;     // [rowsA] rows lda bytes apart
  const char* B;     // [rowsB] rows ldb bytes apart
  size_t lda, ldb;
  int rowsA, rowsB;
  int kbytes;        // of a row (a multiple of 16); split i of `splits` takes ksplit bytes of it
  int ksplit, splits;
  int ti, tj;        // tiles
  // kStats, kGradZ
  const int32_t* labels;
  int v0;            // vocabulary index of A's first row
  float2* part;      // [strips, rowsB] (largest logit, sum of exp against it)
  float* zlab;       // [rowsB]
  const float* lse;
  const float* grad_loss;
  int V;
  char* gn;          // [rowsB, ldgn bytes]
  char* gt;          // [rowsA, ldgt bytes]
  size_t ldgn, ldgt;
  int vpad, npad;    // columns of gn and gt that are written (zeros past the valid ones)
  // kAcc, kStore
  float* acc;        // [splits, rowsB, rowsA]
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
  __shared__ __attribute__((aligned(128))) char lds[ST * STAGE];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wi = wave % WM, wj = wave / WM;
  const int l16 = lane & 15, q = lane >> 4;

  int tile = xcd_tile((int)blockIdx.x, g.ti * g.tj * g.splits);
  const int split = tile / (g.ti * g.tj);
  tile -= split * (g.ti * g.tj);
  const int band = tile / (8 * g.ti), in = tile - band * 8 * g.ti;
  const int bw = min(8, g.tj - band * 8);
  const int i0 = in / bw * BM, j0 = (band * 8 + in % bw) * BN;

  const int kb = split * g.ksplit, kbytes = max(0, min(g.ksplit, g.kbytes - kb));   // a last split may be empty
  const int full = kbytes / kStepBytes, rem = kbytes - full * kStepBytes;
  const int nk = full + (rem > 0);
  const char* A = g.A + (size_t)i0 * g.lda + kb;
  const char* B = g.B + (size_t)j0 * g.ldb + kb;

  // chunk u of this thread: row (u NW + wave) 8 + lane / 8 of the operand (clamped to the last one),
  // stored at chunk lane % 8 and so read from chunk (lane % 8) ^ (row % 8)
  const int lr = lane >> 3, lc = ((lane & 7) ^ lr) * 16;
  uint32_t va[CA], vb[CB];
#pragma unroll
  for (int u = 0; u < CA; ++u) va[u] = (uint32_t)min((u * NW + wave) * 8 + lr, g.rowsA - 1 - i0) * (uint32_t)g.lda + lc;
#pragma unroll
  for (int u = 0; u < CB; ++u) vb[u] = (uint32_t)min((u * NW + wave) * 8 + lr, g.rowsB - 1 - j0) * (uint32_t)g.ldb + lc;

  auto issue = [&](int t) {
    char* dst = lds + (t % ST) * STAGE + wave * 1024;
    const char* a = A + (size_t)t * kStepBytes;
    const char* b = B + (size_t)t * kStepBytes;
    if (t < full) {
#pragma unroll
      for (int u = 0; u < CA; ++u)
        __builtin_amdgcn_global_load_lds((const SPEC_GLOBAL void*)(a + va[u]), (SPEC_LDS void*)(dst + u * NW * 1024), 16,
                                         0, 0);
#pragma unroll
      for (int u = 0; u < CB; ++u)
        __builtin_amdgcn_global_load_lds((const SPEC_GLOBAL void*)(b + vb[u]),
                                         (SPEC_LDS void*)(dst + BM * kStepBytes + u * NW * 1024), 16, 0, 0);
    } else {   // the last step of a row that is no multiple of 128 bytes: zeros behind its end
      const bool on = lc < rem;
      const v4u32 zero = {};
#pragma unroll
      for (int u = 0; u < CA; ++u)
        *reinterpret_cast<v4u32*>(dst + u * NW * 1024 + lane * 16) =
            on ? *reinterpret_cast<const v4u32*>(a + va[u]) : zero;
#pragma unroll
      for (int u = 0; u < CB; ++u)
        *reinterpret_cast<v4u32*>(dst + BM * kStepBytes + u * NW * 1024 + lane * 16) =
            on ? *reinterpret_cast<const v4u32*>(b + vb[u]) : zero;
    }
  };

  f32x4 c[MT][NT] = {};
  const int ra = (wi * MT * 16 + l16) * kStepBytes, rb = BM * kStepBytes + (wj * NT * 16 + l16) * kStepBytes;
#pragma unroll
  for (int t = 0; t < ST - 1; ++t)
    if (t < nk) issue(t);
  for (int t = 0; t < nk; ++t) {
    if (t + ST - 1 <= nk) wait_barrier<(ST - 2) * (CA + CB)>();
    else wait_barrier<0>();
    if (t + ST - 1 < nk) issue(t + ST - 1);   // over the buffer of step t - 1, which every wave has left
    const char* src = lds + (t % ST) * STAGE;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const int ph = ((kk * 4 + q) ^ (lane & 7)) * 16;
      v4u32 a[MT], b[NT];
#pragma unroll
      for (int m = 0; m < MT; ++m) a[m] = *reinterpret_cast<const v4u32*>(src + ra + m * 16 * kStepBytes + ph);
#pragma unroll
      for (int n = 0; n < NT; ++n) b[n] = *reinterpret_cast<const v4u32*>(src + rb + n * 16 * kStepBytes + ph);
#pragma unroll
      for (int m = 0; m < MT; ++m)
#pragma unroll
        for (int n = 0; n < NT; ++n) c[m][n] = mma<ES>(a[m], b[n], c[m][n]);
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
        const int rel = g.labels[j] - iw;   // the lane that holds the label's logit writes it
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
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int j = jw + n * 16;
      const int jc = min(j, g.rowsB - 1);
      const int label = g.labels[jc];
      const float lse = g.lse[jc];
      const bool live = j < g.rowsB && live_row(label, lse, g.V);
      const float s = g.grad_loss[jc];
      const int lab = label - g.v0;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int i = iw + m * 16;
        f32x4 o;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const float p = __builtin_amdgcn_exp2f((c[m][n][x] - lse) * kLog2eF);
          o[x] = (live && i + x < g.rowsA) ? (p - (i + x == lab ? 1.f : 0.f)) * s : 0.f;
        }
        if constexpr (ES == 2) {
          bf16x4 h;
#pragma unroll
          for (int x = 0; x < 4; ++x) h[x] = (__bf16)o[x];
          if (j < g.rowsB && i < g.vpad) *reinterpret_cast<bf16x4*>(g.gn + (size_t)j * g.ldgn + (size_t)i * 2) = h;
          if (j < g.npad)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (i + x < g.rowsA) *reinterpret_cast<__bf16*>(g.gt + (size_t)(i + x) * g.ldgt + (size_t)j * 2) = h[x];
        } else {
          if (j < g.rowsB && i < g.vpad) *reinterpret_cast<f32x4*>(g.gn + (size_t)j * g.ldgn + (size_t)i * 4) = o;
          if (j < g.npad)
#pragma unroll
            for (int x = 0; x < 4; ++x)
              if (i + x < g.rowsA) *reinterpret_cast<float*>(g.gt + (size_t)(i + x) * g.ldgt + (size_t)j * 4) = o[x];
        }
      }
    }
  } else {
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int j = jw + n * 16;
      if (j >= g.rowsB) continue;
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const int i = iw + m * 16;
        if (i >= g.rowsA) continue;   // rowsA is a multiple of 4
        f32x4 o = c[m][n];
        if constexpr (KIND == kAcc) {
          f32x4* p = reinterpret_cast<f32x4*>(g.acc + ((size_t)split * g.rowsB + j) * g.rowsA + i);
          if (g.accumulate) o += *p;
          *p = o;
        } else if constexpr (ES == 2) {
          bf16x4 h;
#pragma unroll
          for (int x = 0; x < 4; ++x) h[x] = (__bf16)o[x];
          *reinterpret_cast<bf16x4*>(g.out + (size_t)j * g.ldo + (size_t)i * 2) = h;
        } else {
          *reinterpret_cast<f32x4*>(g.out + (size_t)j * g.ldo + (size_t)i * 4) = o;
        }
      }
    }
  }
}

// Strips -> lse, loss and status per row: 16 rows per workgroup, 64 threads share a row's strips
// (each a running maximum and fp64 sum), joined in LDS.
constexpr int kCombineThreads = 1024;

__global__ __launch_bounds__(kCombineThreads) void xent_combine_kernel(const float2* part, int strips, int N, int V,
                                                                       const int32_t* labels, const float* zlab,
                                                                       float* loss, float* lse, int32_t* status) {
  __shared__ float sm[64][17];
  __shared__ double ss[64][17];
  const int r = threadIdx.x & 15, h = threadIdx.x >> 4;
  const int n = (int)blockIdx.x * 16 + r, nc = min(n, N - 1);
  float m = -INFINITY;
  double s = 0.0;
  for (int t = h; t < strips; t += 64) {
    const float2 p = part[(size_t)t * N + nc];
    if (p.x > m) {
      s = s * (double)__builtin_amdgcn_exp2f((m - p.x) * kLog2eF) + (double)p.y;
      m = p.x;
    } else {
      s += p.x > -INFINITY ? (double)p.y * (double)__builtin_amdgcn_exp2f((p.x - m) * kLog2eF) : (double)p.y;
    }
  }
  sm[h][r] = m;
  ss[h][r] = s;
  __syncthreads();
  if (h == 0 && n < N) {
    float M = -INFINITY;
    for (int t = 0; t < 64; ++t) M = fmaxf(M, sm[t][r]);
    double S = 0.0;
    for (int t = 0; t < 64; ++t) S += sm[t][r] > -INFINITY ? ss[t][r] * exp((double)sm[t][r] - (double)M) : ss[t][r];
    const bool fin = M < INFINITY && M > -INFINITY && S > 0.0 && S < INFINITY;   // NaN sums fail too
    const double l = (double)M + log(S);
    const int label = labels[n];
    int st = 0;
    if (label < -1 || label >= V) st |= SPEC_REQ_BAD_TOKEN;
    if (label != -1 && !fin) st |= SPEC_REQ_NONFINITE;
    lse[n] = fin ? (float)l : NAN;
    loss[n] = label == -1 ? 0.f : (st ? NAN : (float)(l - (double)zlab[n]));
    if (status) status[n] = st;
  }
}

// out[c][r] = in[r][c], r < R valid and not left out (else 0) for r < rpad; 64 x 64 tiles.
template <int ES>
__global__ __launch_bounds__(256) void xent_transpose_kernel(const char* in, size_t ldi, int R, int C, char* out,
                                                             size_t ldo, int rpad, const int32_t* labels,
                                                             const float* lse, int V) {
  constexpr int EPC = 16 / ES, CPR = 64 / EPC;   // elements per chunk, chunks per tile row
  using E = typename std::conditional<ES == 2, uint16_t, uint32_t>::type;
  __shared__ E t[64][64 + (ES == 2 ? 2 : 1)];
  const int r0 = (int)blockIdx.x * 64, c0 = (int)blockIdx.y * 64, tid = threadIdx.x;
  for (int u = tid; u < 64 * CPR; u += 256) {
    const int r = u / CPR, cc = u % CPR;
    v4u32 v = {};
    const bool on = r0 + r < R && c0 + cc * EPC < C;
    if (on && (!labels || live_row(labels[r0 + r], lse[r0 + r], V)))
      v = *reinterpret_cast<const v4u32*>(in + (size_t)(r0 + r) * ldi + (size_t)(c0 + cc * EPC) * ES);
    const E* e = reinterpret_cast<const E*>(&v);
#pragma unroll
    for (int x = 0; x < EPC; ++x) t[r][cc * EPC + x] = e[x];
  }
  __syncthreads();
  for (int u = tid; u < 64 * CPR; u += 256) {
    const int cc = u / CPR, rc = u % CPR;
    if (c0 + cc < C && r0 + rc * EPC < rpad) {
      v4u32 v;
      E* e = reinterpret_cast<E*>(&v);
#pragma unroll
      for (int x = 0; x < EPC; ++x) e[x] = t[rc * EPC + x][cc];
      *reinterpret_cast<v4u32*>(out + (size_t)(c0 + cc) * ldo + (size_t)(r0 + rc * EPC) * ES) = v;
    }
  }
}

// grad_hidden = the sum of the splits, rounded once; zeros for the rows left out.
template <int ES>
__global__ __launch_bounds__(256) void xent_finish_kernel(const float* acc, int splits, int N, int d, char* out,
                                                          const int32_t* labels, const float* lse, int V) {
  const size_t n4 = (size_t)N * d / 4, t = (size_t)blockIdx.x * 256 + threadIdx.x;
  if (t >= n4) return;
  const int n = (int)(t * 4 / d);
  f32x4 s = {};
  if (live_row(labels[n], lse[n], V))
    for (int i = 0; i < splits; ++i) s += reinterpret_cast<const f32x4*>(acc + (size_t)i * N * d)[t];
  if constexpr (ES == 2) {
    bf16x4 h;
#pragma unroll
    for (int x = 0; x < 4; ++x) h[x] = (__bf16)s[x];
    reinterpret_cast<bf16x4*>(out)[t] = h;
  } else {
    reinterpret_cast<f32x4*>(out)[t] = s;
  }
}

// ---- host -------------------------------------------------------------------

inline int ceil_div(long long a, long long b) { return (int)((a + b - 1) / b); }
inline long long round_to(long long a, long long b) { return (a + b - 1) / b * b; }

// Tile shapes of the product: 256 x 256 (8 waves) when such tiles fill the 256 CUs, 128 x 128 (4 waves,
// two workgroups per CU) below that, 128 x 64 when B has at most 64 rows.
enum { kBig = 0, kMid = 1, kThin = 2 };

inline int pick_tile(long long rowsA, long long rowsB, int splits) {
  if (rowsB <= 64) return kThin;
  return (long long)ceil_div(rowsA, 256) * ceil_div(rowsB, 256) * splits >= 256 ? kBig : kMid;
}
inline int tile_m(int t) { return t == kBig ? 256 : 128; }
inline int tile_n(int t) { return t == kBig ? 256 : t == kMid ? 128 : 64; }
inline int strip_rows(int t) { return t == kBig ? 128 : 64; }

template <int ES, int KIND>
void launch_gemm(GemmArgs& g, int tile, hipStream_t s) {
  g.ti = ceil_div(g.rowsA, tile_m(tile));
  g.tj = ceil_div(g.rowsB, tile_n(tile));
  const dim3 grid((unsigned)(g.ti * g.tj * g.splits));   // within head_fits
  if (tile == kBig)
    hipLaunchKernelGGL((xent_gemm_kernel<ES, 256, 256, 2, 4, 2, KIND>), grid, dim3(512), 0, s, g);
  else if (tile == kMid)
    hipLaunchKernelGGL((xent_gemm_kernel<ES, 128, 128, 2, 2, 2, KIND>), grid, dim3(256), 0, s, g);
  else
    hipLaunchKernelGGL((xent_gemm_kernel<ES, 128, 64, 2, 2, 3, KIND>), grid, dim3(256), 0, s, g);
}

// Every launch's work-items fit the 32-bit grid size of the dispatch packet (tiles below 256 x 256 are
// taken only where fewer than 256 such tiles would do, and contraction splits only below 512 tiles).
bool head_fits(long long N, long long V, long long d) {
  const long long most = 0xffffffffll;
  return (long long)ceil_div(V, 256) * ceil_div(N, 256) * 512 <= most && N * d / 4 + 256 <= most &&
         (long long)ceil_div(V, 256) * ceil_div(d, 256) * 512 <= most;
}

bool head_ok(int N, int V, int d, int dtype) {
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return false;
  if (N < 1 || N > SPEC_MAX_HEAD_ROWS || V < 1 || V > SPEC_MAX_V || d < 1 || d > SPEC_MAX_HEAD_WIDTH) return false;
  return (d * (dtype == SPEC_BF16 ? 2 : 4)) % 16 == 0;
}

// The backward's pieces and its workspace.
struct BackPlan {
  int es, step;          // element size, elements per 128 bytes
  int pieces, vc;        // vocabulary pieces of vc tokens (a multiple of 256; the last may be shorter)
  long long npad;
  int splits, ksplit;    // of the contraction of dH over a piece
  size_t gn, gt, wt, ht, acc;   // bytes
  size_t total() const { return gn + gt + wt + ht + acc; }
};

constexpr long long kPieceBytes = 128ll << 20;   // of G (and of W^T) per piece

BackPlan back_plan(int N, int V, int d, int dtype) {
  BackPlan p{};
  p.es = dtype == SPEC_BF16 ? 2 : 4;
  p.step = kStepBytes / p.es;
  p.npad = round_to(N, p.step);
  const long long widest = N > d ? N : d;
  long long vmax = kPieceBytes / (widest * p.es) / 256 * 256;
  if (vmax < 256) vmax = 256;
  p.pieces = ceil_div(V, vmax);
  p.vc = (int)round_to(ceil_div(V, p.pieces), 256);
  p.pieces = ceil_div(V, p.vc);
  const int tile = N <= 64 ? kThin : kMid;
  const long long tiles = (long long)ceil_div(d, tile_m(tile)) * ceil_div(N, tile_n(tile));
  const int steps = p.vc / p.step;
  long long s = tiles >= 512 ? 1 : 512 / tiles;
  if (s > 16) s = 16;
  if (s > steps / 4) s = steps / 4 > 0 ? steps / 4 : 1;
  p.ksplit = ceil_div(steps, s) * kStepBytes;
  p.splits = ceil_div((long long)p.vc * p.es, p.ksplit);
  p.gn = round256((size_t)N * p.vc * p.es);
  p.gt = round256((size_t)p.vc * p.npad * p.es);
  p.wt = round256((size_t)d * p.vc * p.es);
  p.ht = round256((size_t)d * p.npad * p.es);
  p.acc = round256((size_t)p.splits * N * d * sizeof(float));
  return p;
}

template <int ES>
int32_t run_forward(int N, int V, int d, const void* hidden, const void* weight, const int32_t* labels, float* loss,
                    float* lse, int32_t* status, char* ws, hipStream_t s) {
  const int tile = pick_tile(V, N, 1);
  const int strips = ceil_div(V, tile_m(tile)) * (tile_m(tile) / strip_rows(tile));
  GemmArgs g{};
  g.A = reinterpret_cast<const char*>(weight); g.B = reinterpret_cast<const char*>(hidden);
  g.lda = g.ldb = (size_t)d * ES;
  g.rowsA = V; g.rowsB = N; g.kbytes = d * ES; g.ksplit = g.kbytes; g.splits = 1;
  g.labels = labels; g.V = V;
  g.part = reinterpret_cast<float2*>(ws);
  g.zlab = reinterpret_cast<float*>(ws + round256((size_t)strips * N * sizeof(float2)));
  launch_gemm<ES, kStats>(g, tile, s);
  hipLaunchKernelGGL(xent_combine_kernel, dim3(ceil_div(N, 16)), dim3(kCombineThreads), 0, s, g.part, strips, N, V,
                     labels, g.zlab, loss, lse, status);
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
  const size_t ld = (size_t)d * ES;
  if (grad_weight)
    hipLaunchKernelGGL(xent_transpose_kernel<ES>, dim3(ceil_div(p.npad, 64), ceil_div(d, 64)), dim3(256), 0, s,
                       reinterpret_cast<const char*>(hidden), ld, N, d, ht, (size_t)p.npad * ES, (int)p.npad, labels,
                       lse, V);
  for (int c = 0; c < p.pieces; ++c) {
    const int v0 = c * p.vc, nv = V - v0 < p.vc ? V - v0 : p.vc;
    const int vpad = (int)round_to(nv, p.step);
    const char* w = reinterpret_cast<const char*>(weight) + (size_t)v0 * ld;
    GemmArgs g{};
    g.A = w; g.B = reinterpret_cast<const char*>(hidden);
    g.lda = g.ldb = ld;
    g.rowsA = nv; g.rowsB = N; g.kbytes = d * ES; g.ksplit = g.kbytes; g.splits = 1;
    g.labels = labels; g.V = V; g.v0 = v0; g.lse = lse; g.grad_loss = grad_loss;
    g.gn = gn; g.ldgn = (size_t)p.vc * ES; g.vpad = vpad;
    g.gt = gt; g.ldgt = (size_t)p.npad * ES; g.npad = (int)p.npad;
    launch_gemm<ES, kGradZ>(g, pick_tile(nv, N, 1), s);
    if (grad_hidden) {
      hipLaunchKernelGGL(xent_transpose_kernel<ES>, dim3(ceil_div(vpad, 64), ceil_div(d, 64)), dim3(256), 0, s, w, ld,
                         nv, d, wt, (size_t)p.vc * ES, vpad, nullptr, nullptr, 0);
      GemmArgs h{};
      h.A = wt; h.lda = (size_t)p.vc * ES; h.rowsA = d;
      h.B = gn; h.ldb = (size_t)p.vc * ES; h.rowsB = N;
      h.kbytes = vpad * ES; h.ksplit = p.ksplit; h.splits = p.splits;   // every split is written
      h.acc = acc; h.accumulate = c > 0;
      launch_gemm<ES, kAcc>(h, pick_tile(d, N, h.splits), s);
    }
    if (grad_weight) {
      GemmArgs h{};
      h.A = ht; h.lda = (size_t)p.npad * ES; h.rowsA = d;
      h.B = gt; h.ldb = (size_t)p.npad * ES; h.rowsB = nv;
      h.kbytes = (int)p.npad * ES; h.ksplit = h.kbytes; h.splits = 1;
      h.out = reinterpret_cast<char*>(grad_weight) + (size_t)v0 * ld; h.ldo = ld;
      launch_gemm<ES, kStore>(h, pick_tile(d, nv, 1), s);
    }
  }
  if (grad_hidden)
    hipLaunchKernelGGL(xent_finish_kernel<ES>, dim3(ceil_div((long long)N * d / 4, 256)), dim3(256), 0, s, acc,
                       p.splits, N, d, reinterpret_cast<char*>(grad_hidden), labels, lse, V);
  return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_ERR_HIP;
}

}  // namespace
}  // namespace spec

using namespace spec;

extern "C" size_t spec_head_xent_workspace_size(int32_t N, int32_t V, int32_t d, int32_t dtype) {
  if (!head_ok(N, V, d, dtype)) return 0;
  const int tile = pick_tile(V, N, 1);
  const size_t strips = (size_t)ceil_div(V, tile_m(tile)) * (tile_m(tile) / strip_rows(tile));
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
  if (!head_fits(N, V, d)) return SPEC_ERR_UNSUPPORTED;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  char* ws = reinterpret_cast<char*>(workspace);
  return dtype == SPEC_BF16
             ? run_backward<2>(N, V, d, dtype, hidden, weight, labels, lse, grad_loss, grad_hidden, grad_weight, ws, s)
             : run_backward<4>(N, V, d, dtype, hidden, weight, labels, lse, grad_loss, grad_hidden, grad_weight, ws, s);
}
