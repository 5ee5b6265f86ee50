// The norm in front of the vocabulary head on gfx950, its gradients, and the head's weight in 8 bits.
//
//   h = x + residual;  rstd = 1 / sqrt(mean(h^2) + eps);  y = h rstd w
//   8 bits: amax over each 128 of a row, at least 2^-100; scale = amax / 448; code = e4m3(y 448 / amax)
//   gradients, with xh = h rstd and g = grad_y w:
//     grad_x = rstd (g - xh mean(g xh)) + grad_h;  grad_w = sum over the rows of grad_y xh
//   weight: the same codes with an amax for each block of 128 x 128
//
// All of them are bound by memory: a row is read once into registers (16 values a thread at most, 8 of them in a
// row), and everything else is done there.  16 lanes hold 128 values, one group of the scales: its amax is a
// reduction within a DPP row.  A team of T threads takes a row; a workgroup has 256 threads or one team.
// MI355X, bf16 with a residual: 4352 x 4096 to 8 bits 23-25 us (5.0-5.4 TB/s; a large copy runs at 4.8); 8192 x 4096
// forward 50 us and backward 51 + 5 (5.3 TB/s); weight of 151936 x 4096 to 8 bits 317-322 us (5.8 TB/s).
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <tuple>
#include <utility>

#include "common.hpp"
#include "rowseg.hpp"
#include "spec_verify.h"
#include "xent_plan.hpp"

namespace spec {
namespace {

typedef unsigned int v2u32 __attribute__((ext_vector_type(2)));

constexpr float kCodeMax = 448.f;        // e4m3's largest value
constexpr float kAmaxFloor = 0x1p-100f;  // so that 448 / amax stays in range (and a block of zeros has a scale)
constexpr int kBackThreads = 1 << 18;    // of the backward kernel, at most
constexpr int kSumSlices = 32, kSumCols = 32;

struct NormArgs {
  const void* x;
  const void* residual;
  const void* w;
  void* h;
  void* y;          // in the inputs' type, or
  uint8_t* codes;   // [N, d]
  float* scales;    // [N, groups]
  float* rstd;
  int N, d, groups;
  float eps;
};

struct BackArgs {
  const void* grad_y;
  const void* h;
  const void* w;
  const float* rstd;
  const void* grad_h;
  void* grad_x;
  float* part;      // [gridDim.x, d], or NULL
  int N, d;
};

// 16 bytes at an address of that alignment: rows that are no multiple of 16 bytes start anywhere.
template <int ALIGN>
struct __attribute__((packed, aligned(ALIGN))) Piece {
  v4u32 v;
};

// 8 consecutive values of a row from index c; zeros past d.  VEC: the rows are multiples of 16 bytes.
template <bool BF16, bool VEC>
__device__ __forceinline__ void load8(const void* p, size_t row, int c, int d, float (&v)[8]) {
  constexpr int ES = BF16 ? 2 : 4;
  const char* src = reinterpret_cast<const char*>(p) + (row + c) * ES;
#pragma unroll
  for (int x = 0; x < 8; ++x) v[x] = 0.f;
  if (c + 8 <= d || (VEC && !BF16 && c + 4 <= d)) {
    const v4u32 t = reinterpret_cast<const Piece<VEC ? 16 : ES>*>(src)->v;
    if constexpr (BF16) {
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        v[2 * x] = bf16_lo(t[x]);
        v[2 * x + 1] = bf16_hi(t[x]);
      }
    } else {
#pragma unroll
      for (int x = 0; x < 4; ++x) v[x] = __uint_as_float(t[x]);
      if (!VEC || c + 8 <= d) {
        const v4u32 u = reinterpret_cast<const Piece<VEC ? 16 : ES>*>(src + 16)->v;
#pragma unroll
        for (int x = 0; x < 4; ++x) v[4 + x] = __uint_as_float(u[x]);
      }
    }
  } else if (!VEC) {
#pragma unroll
    for (int x = 0; x < 7; ++x)
      if (c + x < d) v[x] = load_elem<BF16>(src, x);
  }
}

__device__ __forceinline__ uint32_t bf16_bits(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }

template <bool BF16, bool VEC>
__device__ __forceinline__ void store8(void* p, size_t row, int c, int d, const float (&v)[8]) {
  constexpr int ES = BF16 ? 2 : 4;
  char* dst = reinterpret_cast<char*>(p) + (row + c) * ES;
  if (c + 8 <= d || (VEC && !BF16 && c + 4 <= d)) {
    v4u32 t;
    if constexpr (BF16) {
#pragma unroll
      for (int x = 0; x < 4; ++x) t[x] = bf16_bits(v[2 * x]) | bf16_bits(v[2 * x + 1]) << 16;
      reinterpret_cast<Piece<VEC ? 16 : ES>*>(dst)->v = t;
    } else {
#pragma unroll
      for (int x = 0; x < 4; ++x) t[x] = __float_as_uint(v[x]);
      reinterpret_cast<Piece<VEC ? 16 : ES>*>(dst)->v = t;
      if (!VEC || c + 8 <= d) {
#pragma unroll
        for (int x = 0; x < 4; ++x) t[x] = __float_as_uint(v[4 + x]);
        reinterpret_cast<Piece<VEC ? 16 : ES>*>(dst + 16)->v = t;
      }
    }
  } else if (!VEC) {
#pragma unroll
    for (int x = 0; x < 7; ++x) {
      if (c + x >= d) break;
      if constexpr (BF16) reinterpret_cast<uint16_t*>(dst)[x] = (uint16_t)bf16_bits(v[x]);
      else reinterpret_cast<float*>(dst)[x] = v[x];
    }
  }
}

constexpr int kWorkgroup = 256;   // threads, where a team has fewer
constexpr int teams(int T) { return T < kWorkgroup ? kWorkgroup / T : 1; }

// Sum over the thread's team, in wave order; `sh` holds a word per wave of the workgroup and is free until the next but
// one call where the callers alternate between two.
template <int T>
__device__ __forceinline__ float team_sum(float x, float* sh) {
  x = wave_reduce(x, [](float a, float b) { return a + b; });
  if constexpr (T == SPEC_WAVE) return x;
  constexpr int NW = T / SPEC_WAVE;
  const int wave = threadIdx.x >> 6;
  if ((threadIdx.x & 63) == 0) sh[wave] = x;
  __syncthreads();
  sh += wave / NW * NW;
  float s = sh[0];
#pragma unroll
  for (int w = 1; w < NW; ++w) s += sh[w];
  return s;
}

// Largest magnitude as its bits: NaN above infinity above every finite value.
template <int T>
__device__ __forceinline__ uint32_t team_amax(uint32_t x, float* sh) {
  x = wave_reduce(x, [](uint32_t a, uint32_t b) { return max(a, b); });
  if constexpr (T == SPEC_WAVE) return x;
  constexpr int NW = T / SPEC_WAVE;
  const int wave = threadIdx.x >> 6;
  uint32_t* s = reinterpret_cast<uint32_t*>(sh);
  if ((threadIdx.x & 63) == 0) s[wave] = x;
  __syncthreads();
  s += wave / NW * NW;
  uint32_t m = s[0];
#pragma unroll
  for (int w = 1; w < NW; ++w) m = max(m, s[w]);
  return m;
}

__device__ __forceinline__ uint32_t magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// Four values in [-448 (1 + 2^-23), 448 (1 + 2^-23)] (or NaN) as e4m3, ties to even.
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
}

template <bool BF16, bool VEC, bool Q8, int T, int K>
__global__ __launch_bounds__(T * teams(T)) void norm_kernel(NormArgs a) {
  __shared__ float sh[4][T * teams(T) / SPEC_WAVE];
  const int tid = threadIdx.x % T, d = a.d, n = (int)blockIdx.x * teams(T) + threadIdx.x / T;
  const bool live = n < a.N;   // past the last row: its values again, nothing stored
  const size_t row = (size_t)min(n, a.N - 1) * d;
  float v[K][8], w[K][8];
#pragma unroll
  for (int k = 0; k < K; ++k) load8<BF16, VEC>(a.x, row, (k * T + tid) * 8, d, v[k]);
  if (a.residual) {
    float r[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k) load8<BF16, VEC>(a.residual, row, (k * T + tid) * 8, d, r[k]);
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int x = 0; x < 8; ++x) v[k][x] += r[k][x];
  }
#pragma unroll
  for (int k = 0; k < K; ++k) load8<BF16, VEC>(a.w, 0, (k * T + tid) * 8, d, w[k]);
  // the norm is taken of the sum in fp32; only what is stored of it is rounded
  if (a.h && live)
#pragma unroll
    for (int k = 0; k < K; ++k) store8<BF16, VEC>(a.h, row, (k * T + tid) * 8, d, v[k]);
  float ss = 0.f;
#pragma unroll
  for (int k = 0; k < K; ++k)
#pragma unroll
    for (int x = 0; x < 8; ++x) ss += v[k][x] * v[k][x];
  ss = team_sum<T>(ss, sh[0]);
  float rs = 1.f / sqrtf(ss / (float)d + a.eps), rstd = rs;
  bool off = !(ss >= 0x1p-90f && ss <= 0x1p120f);
  if (T == SPEC_WAVE ? off : __syncthreads_or(off)) {
    // the squares left fp32's range (or nearly): taken again of the row scaled by a power of two
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int x = 0; x < 8; ++x) m = max(m, magnitude(v[k][x]));
    m = team_amax<T>(m, sh[1]);
    off = off && m != 0 && m < 0x7f800000u;
    const int e = off ? ilogbf(__uint_as_float(m)) : 0;
    float sq = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const float y = ldexpf(v[k][x], -e);
        sq += y * y;
        if (off) v[k][x] = y;
      }
    sq = team_sum<T>(sq, sh[2]);
    if (off) {
      const double r = 1.0 / sqrt(ldexp((double)sq / d, 2 * e) + (double)a.eps);
      rs = (float)ldexp(r, e);
      rstd = (float)r;
    }
  }
  if (!live) return;
  if (a.rstd && tid == 0) a.rstd[n] = rstd;
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int c = (k * T + tid) * 8;
#pragma unroll
    for (int x = 0; x < 8; ++x) v[k][x] = v[k][x] * rs * w[k][x];
    if constexpr (!Q8) {
      store8<BF16, VEC>(a.y, row, c, d, v[k]);
    } else {
      uint32_t m = __float_as_uint(kAmaxFloor);
#pragma unroll
      for (int x = 0; x < 8; ++x)
        if (c < d) m = max(m, magnitude(v[k][x]));   // past the row: 0, but 0 * inf where the row's norm is
      auto mx = [](uint32_t p, uint32_t q) { return max(p, q); };
      m = mx(m, dpp_move<dpp::kQuadXor1>(m, m));
      m = mx(m, dpp_move<dpp::kQuadXor2>(m, m));
      m = mx(m, dpp_move<dpp::kRowHalfMirror>(m, m));
      m = mx(m, dpp_move<dpp::kRowMirror>(m, m));
      const float amax = __uint_as_float(m), r = kCodeMax / amax;
      if (c < d) {
        v2u32 q;
        q.x = codes4(v[k][0] * r, v[k][1] * r, v[k][2] * r, v[k][3] * r);
        q.y = codes4(v[k][4] * r, v[k][5] * r, v[k][6] * r, v[k][7] * r);
        *reinterpret_cast<v2u32*>(a.codes + row + c) = q;
        if ((tid & 15) == 0) a.scales[(size_t)n * a.groups + (c >> 7)] = amax / kCodeMax;
      }
    }
  }
}

// Every gridDim.x-th group of a row per team; the weight and its gradient's share stay in registers, and the teams'
// shares are added at the end.
template <bool BF16, bool VEC, int T, int K>
__global__ __launch_bounds__(T * teams(T)) void norm_backward_kernel(BackArgs a) {
  constexpr int TEAMS = teams(T);
  __shared__ float sh[2][T * TEAMS / SPEC_WAVE];
  __shared__ float share[TEAMS > 1 ? TEAMS - 1 : 1][TEAMS > 1 ? 8 * K * T : 1];
  const int tid = threadIdx.x % T, team = threadIdx.x / T, d = a.d;
  float w[K][8], dw[K][8] = {};
#pragma unroll
  for (int k = 0; k < K; ++k) load8<BF16, VEC>(a.w, 0, (k * T + tid) * 8, d, w[k]);
  int turn = 0;
  for (int n0 = (int)blockIdx.x * TEAMS; n0 < a.N; n0 += (int)gridDim.x * TEAMS, turn ^= 1) {
    const int n = n0 + team;
    const bool live = n < a.N;
    const size_t row = (size_t)min(n, a.N - 1) * d;
    const float rstd = a.rstd[min(n, a.N - 1)];
    float gy[K][8], xh[K][8], gh[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      load8<BF16, VEC>(a.grad_y, row, (k * T + tid) * 8, d, gy[k]);
      load8<BF16, VEC>(a.h, row, (k * T + tid) * 8, d, xh[k]);
      // unaligned: behind the sum, or the registers do not do
      if (VEC && a.grad_h) load8<BF16, VEC>(a.grad_h, row, (k * T + tid) * 8, d, gh[k]);
    }
    float dot = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        xh[k][x] *= rstd;
        if (TEAMS == 1 || live) dw[k][x] += gy[k][x] * xh[k][x];
        gy[k][x] *= w[k][x];
        dot += gy[k][x] * xh[k][x];
      }
    dot = team_sum<T>(dot, sh[turn]) / (float)d;
    if (TEAMS > 1 && !live) continue;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (!VEC && a.grad_h) load8<BF16, VEC>(a.grad_h, row, (k * T + tid) * 8, d, gh[k]);
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        gy[k][x] = rstd * (gy[k][x] - xh[k][x] * dot);
        if (a.grad_h) gy[k][x] += gh[k][x];
      }
      store8<BF16, VEC>(a.grad_x, row, (k * T + tid) * 8, d, gy[k]);
    }
  }
  if (!a.part) return;
  if constexpr (TEAMS > 1) {
    if (team > 0)
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int x = 0; x < 8; ++x) share[team - 1][(k * 8 + x) * T + tid] = dw[k][x];
    __syncthreads();
    if (team > 0) return;
#pragma unroll
    for (int q = 0; q < TEAMS - 1; ++q)
#pragma unroll
      for (int k = 0; k < K; ++k)
#pragma unroll
        for (int x = 0; x < 8; ++x) dw[k][x] += share[q][(k * 8 + x) * T + tid];
  }
#pragma unroll
  for (int k = 0; k < K; ++k) store8<false, VEC>(a.part, (size_t)blockIdx.x * d, (k * T + tid) * 8, d, dw[k]);
}

// grad_w: the workgroups' shares in order, in fp64, rounded once.
template <bool BF16>
__global__ __launch_bounds__(kSumSlices* kSumCols) void norm_weight_kernel(const float* part, int P, int d, void* out) {
  __shared__ double sh[kSumSlices][kSumCols];
  const int s = threadIdx.x / kSumCols, c = threadIdx.x % kSumCols, col = blockIdx.x * kSumCols + c;
  double sum = 0.0;
  if (col < d)
#pragma unroll 8
    for (int p = s; p < P; p += kSumSlices) sum += (double)part[(size_t)p * d + col];
  sh[s][c] = sum;
  __syncthreads();
  if (s == 0 && col < d) {
#pragma unroll
    for (int q = 1; q < kSumSlices; ++q) sum += sh[q][c];
    if constexpr (BF16) reinterpret_cast<uint16_t*>(out)[col] = (uint16_t)bf16_bits((float)sum);
    else reinterpret_cast<float*>(out)[col] = (float)sum;
  }
}

// A block of 128 x 128 per workgroup: 16 lanes take 128 columns of a row, 16 rows at a time.
template <bool BF16>
__global__ __launch_bounds__(256) void quantize_kernel(const void* w, int V, int d, int groups, uint8_t* codes,
                                                       float* scales) {
  __shared__ float sh[4];
  const int tid = threadIdx.x, g = blockIdx.x, c = g * 128 + (tid & 15) * 8;
  const int r0 = blockIdx.y * 128 + (tid >> 4);
  float v[8][8];
  uint32_t m = __float_as_uint(kAmaxFloor);
#pragma unroll
  for (int u = 0; u < 8; ++u) load8<BF16, true>(w, (size_t)min(r0 + 16 * u, V - 1) * d, c, d, v[u]);
#pragma unroll
  for (int u = 0; u < 8; ++u)
#pragma unroll
    for (int x = 0; x < 8; ++x) m = max(m, magnitude(v[u][x]));
  const float amax = __uint_as_float(team_amax<256>(m, sh));
  // The code nearest to w 448 / amax, both scaled to amax in [1, 2): the product with the reciprocal, corrected once.
  // Quotients of two bf16 values often lie halfway between two codes, where the last bit decides; else they are further
  // from there than fp32's rounding.  Quotients of fp32 values can lie closer, and are off by up to 1.5 units here (448 w is
  // rounded): those within 2 units of halfway (19 zero bits) are taken again with lo, what 448 w lost.  The sign of what is
  // then left of 448 w says on which side of q the quotient is (the remainders are exact as far as their sign needs), and of
  // the two fp32 values around it the odd one, which is never halfway between codes, rounds as the quotient does.
  const int e = ilogbf(amax);
  const float as = ldexpf(amax, -e), r = kCodeMax / as;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    float q[8];
    bool near = false;
#pragma unroll
    for (int x = 0; x < 8; ++x) {
      const float ws = ldexpf(v[u][x], -e), p = ws * r;
      q[x] = fmaf(fmaf(-p, as, ws * kCodeMax), 1.f / as, p);
      near |= ((__float_as_uint(q[x]) + 2u) & 0x7ffffu) <= 4u;
    }
    if (!BF16 && near && c < d)
#pragma unroll
      for (int x = 0; x < 8; ++x) {
        const float ws = ldexpf(v[u][x], -e), hi = ws * kCodeMax, lo = fmaf(ws, kCodeMax, -hi);
        q[x] = fmaf(fmaf(-q[x], as, hi) + lo, 1.f / as, q[x]);
        const float rest = fmaf(-q[x], as, hi) + lo;
        const uint32_t b = __float_as_uint(q[x]), past = (__float_as_uint(rest) ^ b) >> 31;
        if (rest != 0.f) q[x] = __uint_as_float((b - past) | 1u);
      }
    if (r0 + 16 * u < V && c < d)
      *reinterpret_cast<v2u32*>(codes + (size_t)(r0 + 16 * u) * d + c) =
          v2u32{codes4(q[0], q[1], q[2], q[3]), codes4(q[4], q[5], q[6], q[7])};
  }
  if (tid == 0) scales[(size_t)blockIdx.y * groups + g] = amax / kCodeMax;
}

// ---- host -------------------------------------------------------------------

// Threads and vectors per thread of a row of d values: 16 values a thread, or 8 where a wave holds the row so.
template <class F>
void with_shape(int d, F f) {
  if (d <= 512) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 1>{});
  else if (d <= 1024) f(std::integral_constant<int, 64>{}, std::integral_constant<int, 2>{});
  else if (d <= 2048) f(std::integral_constant<int, 128>{}, std::integral_constant<int, 2>{});
  else if (d <= 4096) f(std::integral_constant<int, 256>{}, std::integral_constant<int, 2>{});
  else if (d <= 8192) f(std::integral_constant<int, 512>{}, std::integral_constant<int, 2>{});
  else f(std::integral_constant<int, 1024>{}, std::integral_constant<int, 2>{});
}

template <class F>
void with_type(int dtype, bool vec, F f) {
  if (dtype == SPEC_BF16) {
    if (vec) f(std::true_type{}, std::true_type{});
    else f(std::true_type{}, std::false_type{});
  } else {
    if (vec) f(std::false_type{}, std::true_type{});
    else f(std::false_type{}, std::false_type{});
  }
}

bool norm_ok(int N, int d, int dtype) {
  return (dtype == SPEC_F32 || dtype == SPEC_BF16) && N >= 1 && N <= SPEC_MAX_HEAD_ROWS && d >= 1 &&
         d <= SPEC_MAX_HEAD_WIDTH;
}

bool vector_rows(int d, int dtype) { return d * (dtype == SPEC_BF16 ? 2 : 4) % 16 == 0; }

// Workgroups of the backward kernel: what its rows need, at most kBackThreads threads of them.  With fewer the memory is
// not kept busy, with more the weight's share of each (d fp32) is written and read for fewer rows: 8192 x 4096 bf16 at
// 512, 1024 and 2048 workgroups of 256 threads 77, 54 and 63 us; 2048 x 8192 at 256, 512 and 1024 of 512 threads
// 33, 29 and 35; 2048 x 16384 at 128, 256 and 512 of 1024 threads 89, 58 and 65.  (fp32 rows do with fewer: 8192 x 4096
// at 256 and 1024 98 and 105 us, 8192 x 2048 at 512 and 1024 45 and 47.)
int back_groups(int N, int d) {
  int groups = 0;
  with_shape(d, [&](auto T, auto) {
    constexpr int rows = teams(T()), most = kBackThreads / (T() * rows);
    groups = ceil_div(N, rows);
    if (groups > most) groups = most;
  });
  return groups;
}

int32_t launched() { return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_ERR_HIP; }

}  // namespace
}  // namespace spec

using namespace spec;

extern "C" int32_t spec_head_norm(int32_t N, int32_t d, int32_t dtype, const void* x, const void* residual,
                                  const void* weight, float eps, void* h_out, void* y_out, uint8_t* codes_out,
                                  float* scales_out, float* rstd_out, void* stream) {
  if (!norm_ok(N, d, dtype) || !(eps >= 0.f) || !(eps < INFINITY)) return SPEC_ERR_INVALID_ARG;
  if (!x || !weight || (residual && !h_out) || (!y_out == !codes_out) || (!codes_out != !scales_out))
    return SPEC_ERR_INVALID_ARG;
  for (const void* p : {x, residual, weight, (const void*)h_out, (const void*)y_out, (const void*)codes_out})
    if (!aligned16(p)) return SPEC_ERR_INVALID_ARG;
  if (codes_out && d % 16) return SPEC_ERR_INVALID_ARG;
  const size_t n = (size_t)N * d, bytes = n * (dtype == SPEC_BF16 ? 2 : 4), wbytes = bytes / N;
  const size_t groups = (size_t)ceil_div(d, 128), sbytes = N * groups * sizeof(float);
  // a row is read whole before anything of it is written: h and y may be x or the residual themselves
  for (auto [p, m, same] : {std::tuple<const void*, size_t, bool>{h_out, bytes, true}, {y_out, bytes, true},
                            {codes_out, n, false}, {scales_out, sbytes, false}, {rstd_out, N * sizeof(float), false}}) {
    if (!(same && p == x) && overlap(p, m, x, bytes)) return SPEC_ERR_INVALID_ARG;
    if (!(same && p == residual) && overlap(p, m, residual, bytes)) return SPEC_ERR_INVALID_ARG;
    if (overlap(p, m, weight, wbytes)) return SPEC_ERR_INVALID_ARG;
  }
  const std::pair<const void*, size_t> outs[] = {{h_out, bytes}, {y_out, bytes}, {codes_out, n}, {scales_out, sbytes},
                                                 {rstd_out, N * sizeof(float)}};
  for (int i = 0; i < 5; ++i)
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i].first, outs[i].second, outs[j].first, outs[j].second)) return SPEC_ERR_INVALID_ARG;
  const NormArgs a{x, residual, weight, h_out, y_out, codes_out, scales_out, rstd_out, N, d, (int)groups, eps};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  with_shape(d, [&](auto T, auto K) {
    with_type(dtype, vector_rows(d, dtype), [&](auto BF, auto VEC) {
      constexpr int rows = teams(T());
      const dim3 grid(ceil_div(N, rows)), block(T() * rows);
      if (!codes_out)
        hipLaunchKernelGGL((norm_kernel<BF(), VEC(), false, T(), K()>), grid, block, 0, s, a);
      else if constexpr (VEC())   // multiples of 16 values
        hipLaunchKernelGGL((norm_kernel<BF(), true, true, T(), K()>), grid, block, 0, s, a);
    });
  });
  return launched();
}

extern "C" size_t spec_head_norm_backward_workspace_size(int32_t N, int32_t d) {
  return norm_ok(N, d, SPEC_F32) ? round256((size_t)back_groups(N, d) * round_to(d, 4) * sizeof(float)) : 0;
}

extern "C" int32_t spec_head_norm_backward(int32_t N, int32_t d, int32_t dtype, const void* grad_y, const void* h,
                                           const void* weight, const float* rstd, const void* grad_h, void* grad_x,
                                           void* grad_weight, void* workspace, size_t workspace_bytes, void* stream) {
  if (!norm_ok(N, d, dtype)) return SPEC_ERR_INVALID_ARG;
  if (!grad_y || !h || !weight || !rstd || !grad_x) return SPEC_ERR_INVALID_ARG;
  for (const void* p : {grad_y, h, weight, grad_h, (const void*)grad_x, (const void*)grad_weight})
    if (!aligned16(p)) return SPEC_ERR_INVALID_ARG;
  if (grad_weight && (!workspace || !aligned256(workspace) || workspace_bytes < spec_head_norm_backward_workspace_size(N, d)))
    return SPEC_ERR_WORKSPACE;
  const size_t bytes = (size_t)N * d * (dtype == SPEC_BF16 ? 2 : 4), wbytes = bytes / N;
  for (const void* p : {grad_y, h, grad_h})   // a row is read before its gradient is written
    if (p != grad_x && overlap(grad_x, bytes, p, bytes)) return SPEC_ERR_INVALID_ARG;
  if (overlap(grad_x, bytes, weight, wbytes) || overlap(grad_x, bytes, rstd, N * sizeof(float)) ||
      overlap(grad_x, bytes, grad_weight, wbytes))
    return SPEC_ERR_INVALID_ARG;
  for (auto [p, m] : {std::pair<const void*, size_t>{grad_y, bytes}, {h, bytes}, {grad_h, bytes}, {weight, wbytes},
                      {rstd, N * sizeof(float)}})
    if (overlap(grad_weight, wbytes, p, m)) return SPEC_ERR_INVALID_ARG;
  const int P = back_groups(N, d);
  const BackArgs a{grad_y, h, weight, rstd, grad_h, grad_x, grad_weight ? reinterpret_cast<float*>(workspace) : nullptr,
                   N, d};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  with_shape(d, [&](auto T, auto K) {
    with_type(dtype, vector_rows(d, dtype), [&](auto BF, auto VEC) {
      hipLaunchKernelGGL((norm_backward_kernel<BF(), VEC(), T(), K()>), dim3(P), dim3(T() * teams(T())), 0, s, a);
    });
  });
  if (grad_weight) {
    const dim3 grid(ceil_div(d, kSumCols)), block(kSumSlices * kSumCols);
    if (dtype == SPEC_BF16) hipLaunchKernelGGL(norm_weight_kernel<true>, grid, block, 0, s, a.part, P, d, grad_weight);
    else hipLaunchKernelGGL(norm_weight_kernel<false>, grid, block, 0, s, a.part, P, d, grad_weight);
  }
  return launched();
}

extern "C" int32_t spec_head_quantize(int32_t V, int32_t d, int32_t dtype, const void* weight, uint8_t* codes_out,
                                      float* scales_out, void* stream) {
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (V < 1 || V > SPEC_MAX_V || d < 16 || d > SPEC_MAX_HEAD_WIDTH || d % 16) return SPEC_ERR_INVALID_ARG;
  if (!weight || !codes_out || !scales_out || !aligned16(weight) || !aligned16(codes_out)) return SPEC_ERR_INVALID_ARG;
  const size_t n = (size_t)V * d, bytes = n * (dtype == SPEC_BF16 ? 2 : 4);
  const size_t sbytes = (size_t)ceil_div(V, 128) * ceil_div(d, 128) * sizeof(float);
  if (overlap(codes_out, n, weight, bytes) || overlap(scales_out, sbytes, weight, bytes) ||
      overlap(codes_out, n, scales_out, sbytes))
    return SPEC_ERR_INVALID_ARG;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const dim3 grid(ceil_div(d, 128), ceil_div(V, 128));
  if (dtype == SPEC_BF16)
    hipLaunchKernelGGL(quantize_kernel<true>, grid, dim3(256), 0, s, weight, V, d, (int)grid.x, codes_out, scales_out);
  else
    hipLaunchKernelGGL(quantize_kernel<false>, grid, dim3(256), 0, s, weight, V, d, (int)grid.x, codes_out, scales_out);
  return launched();
}
