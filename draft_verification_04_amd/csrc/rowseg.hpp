// One segment of a logit row held in the registers of a workgroup (training kernels).
//
// A row's 16-byte body is cut into segments of at most kSegThreads * kSegVecs vectors (64 KB), one
// workgroup each; every thread issues its kSegVecs loads at once and keeps the vectors, so a segment
// is read from memory once however many passes its kernel makes over it.  The elements before the
// first and after the last whole vector (at most 7 + 7, rows that do not start or end on a 16-byte
// boundary) belong to segment 0, one per thread.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.hpp"
#include "spec_verify.h"

namespace spec {

constexpr int kSegThreads = 512;
constexpr int kSegWaves = kSegThreads / SPEC_WAVE;
constexpr int kSegVecs = 8;   // 16-byte vectors per thread: 32 registers, 8 waves per SIMD
constexpr double kLog2eSeg = 1.44269504088896340736;

inline int row_segments(int V, int dtype) {
  const int vecs = V / (dtype == SPEC_BF16 ? 8 : 4);
  const int cap = kSegThreads * kSegVecs;
  return vecs <= cap ? 1 : (vecs + cap - 1) / cap;
}

template <bool BF16>
struct RowSeg {
  static constexpr int ES = BF16 ? 2 : 4;
  static constexpr int EPV = 16 / ES;
  static constexpr uint32_t kNegInf = BF16 ? 0xff80ff80u : 0xff800000u;
  int head, tail0;   // elements before the body; first element after it
  int vb, ve;        // this segment's vectors of the body
  int nx;            // scalar elements of this segment (head and tail; segment 0 only)

  __device__ __forceinline__ RowSeg(const char* row, int V, int seg, int nseg) {
    const unsigned mis = (unsigned)(reinterpret_cast<uintptr_t>(row) & 15u);
    head = min((int)(((16u - mis) & 15u) / ES), V);
    const int nv = (V - head) / EPV;
    tail0 = head + nv * EPV;
    vb = (int)((long long)nv * seg / nseg);
    ve = (int)((long long)nv * (seg + 1) / nseg);
    nx = seg == 0 ? head + (V - tail0) : 0;
  }
  // token id of element e of body vector v, and of the thread's scalar element
  __device__ __forceinline__ int id_of(int v, int e) const { return head + v * EPV + e; }
  __device__ __forceinline__ int id_of_scalar(int t) const { return t < head ? t : tail0 + (t - head); }
  // the thread's vectors (-inf past the segment); loads are issued together, clamped in bounds
  __device__ __forceinline__ void load(const char* row, uint4 (&d)[kSegVecs]) const {
    const uint4* vp = reinterpret_cast<const uint4*>(row + (size_t)head * ES);
#pragma unroll
    for (int j = 0; j < kSegVecs; ++j) {
      d[j] = make_uint4(kNegInf, kNegInf, kNegInf, kNegInf);
      if (vb + j * kSegThreads < ve)
        d[j] = load_nt(vp + min(vb + j * kSegThreads + (int)threadIdx.x, ve - 1));
    }
  }
  __device__ __forceinline__ void mask(uint4 (&d)[kSegVecs]) const {
#pragma unroll
    for (int j = 0; j < kSegVecs; ++j)
      if (vb + j * kSegThreads + (int)threadIdx.x >= ve) d[j] = make_uint4(kNegInf, kNegInf, kNegInf, kNegInf);
  }
  // the thread's vector j read once more
  __device__ __forceinline__ uint4 reload(const char* row, int j) const {
    const int v = vb + j * kSegThreads + (int)threadIdx.x;
    return v < ve ? reinterpret_cast<const uint4*>(row + (size_t)head * ES)[v]
                  : make_uint4(kNegInf, kNegInf, kNegInf, kNegInf);
  }
  __device__ __forceinline__ float load_scalar(const char* row) const {
    return (int)threadIdx.x < nx ? load_elem<BF16>(row, id_of_scalar(threadIdx.x)) : -INFINITY;
  }
  static __device__ __forceinline__ void unpack(const uint4& d, float (&z)[EPV]) {
    const uint32_t w[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if constexpr (BF16) {
        z[2 * q] = bf16_lo(w[q]);
        z[2 * q + 1] = bf16_hi(w[q]);
      } else {
        z[q] = __uint_as_float(w[q]);
      }
    }
  }
};

// The vectors as values the compiler knows nothing about: a second pass over them unpacks them again
// instead of keeping the first pass's unpacked values in registers (twice as many).
__device__ __forceinline__ void forget(uint4 (&d)[kSegVecs]) {
#pragma unroll
  for (int j = 0; j < kSegVecs; ++j) asm volatile("" : "+v"(d[j].x), "+v"(d[j].y), "+v"(d[j].z), "+v"(d[j].w));
}

// log2(e) / T as a float pair, c_hi toward zero and c_lo > 0 (so that a logit of -inf gives an
// exponent of -inf, never NaN); finite for every T > 0 (T towards 0 is the argmax).
__device__ __forceinline__ void split_scale(float T, float& c_hi, float& c_lo) {
  const double c = fmin(kLog2eSeg / (double)T, 3.4028234663852886e38);
  c_hi = __double2float_rz(c);
  c_lo = fmaxf((float)(c - (double)c_hi), 1.4e-45f);
}

// A thread's running sum of exp(z / T) as S 2^M.  M is an integer that only rises, so a rescale is an
// exact power of two, and the exponent z c - M is formed with one rounding at its own size:
// fma(z, c_lo, fma(z, c_hi, -M)).  A vector's sum past 2^32 (NaN included) takes the slow branch: M
// moves up to the vector's largest exponent.  `odd` is set where that cannot be held (NaN, +inf, or an
// exponent past 2^22, whose neighbours an fp32 reference no longer tells apart): the segment is then
// summed again by exp_term.
struct RunningSum {
  float M, S;
  int odd;
};

constexpr float kWideExponent = 0x1p22f;

template <int N>
__device__ __forceinline__ float exp_sum(const float (&z)[N], float c_hi, float c_lo, float M) {
  float e[N];
#pragma unroll
  for (int j = 0; j < N; ++j) e[j] = __builtin_amdgcn_exp2f(fmaf(z[j], c_lo, fmaf(z[j], c_hi, -M)));
#pragma unroll
  for (int w = 1; w < N; w <<= 1)
#pragma unroll
    for (int j = 0; j + w < N; j += 2 * w) e[j] += e[j + w];
  return e[0];
}

template <int N>
__device__ __forceinline__ void add_terms(RunningSum& r, const float (&z)[N], float c_hi, float c_lo) {
  float s = exp_sum<N>(z, c_hi, c_lo, r.M);
  if (!(s <= 0x1p32f)) {
    float vm = z[0];
#pragma unroll
    for (int j = 1; j < N; ++j) vm = fmaxf(vm, z[j]);
    const float mc = ceilf(vm * c_hi);
    s = 0.f;
    if (!(fabsf(mc) < kWideExponent)) {
      r.odd = 1;
    } else {
      if (mc > r.M) {
        const float d = r.M - mc;
        r.S = d < -126.f ? 0.f : ldexpf(r.S, (int)d);
        r.M = mc;
      }
      s = exp_sum<N>(z, c_hi, c_lo, r.M);
      if (!(s <= 0x1p32f)) {   // a NaN beside finite values
        r.odd = 1;
        s = 0.f;
      }
    }
  }
  r.S += s;
}

constexpr float kNoReference = -0x1p24f;   // below every exponent that is summed: the first term raises it

// exp2((z - m) c) against the segment's largest value m: the difference first, so that it, not the
// value, sets the rounding, whatever the values' size.
__device__ __forceinline__ float exp_term(float z, float m, float c_hi, float c_lo) {
  const float dz = z - m;
  return __builtin_amdgcn_exp2f(fmaf(dz, c_lo, dz * c_hi));
}

// A segment's sum of exp(z / T): sum * 2^ref, fp64.
struct SegSum {
  double sum, ref;
};

// Scratch of segment_sum.
struct SegSumShared {
  double s[kSegWaves];
  float m[kSegWaves];
  int odd[kSegWaves];
};

// The workgroup's sum (and whether a NaN or +inf was among the values) from its threads' running sums;
// every thread gets the result.  again(j) reads the thread's vector j once more (-inf where there is
// none) and x is its scalar: used only when a sum was odd.
template <bool BF16, class Again>
__device__ __forceinline__ SegSum segment_sum(SegSumShared& sh, const RunningSum& r, Again again, float x, float c_hi,
                                              float c_lo, int& bad) {
  using Seg = RowSeg<BF16>;
  const int wave = (int)threadIdx.x >> 6, lane = (int)threadIdx.x & 63;
  const float wm = wave_max(r.M);
  const double ws = wave_sum(ldexp((double)r.S, (int)fmaxf(r.M - wm, -2000.f)));
  const int wo = __ballot(r.odd) != 0;
  if (lane == 0) {
    sh.s[wave] = ws;
    sh.m[wave] = wm;
    sh.odd[wave] = wo;
  }
  __syncthreads();
  float M = sh.m[0];
  int odd = sh.odd[0];
#pragma unroll
  for (int w = 1; w < kSegWaves; ++w) {
    M = fmaxf(M, sh.m[w]);
    odd |= sh.odd[w];
  }
  SegSum t{0.0, (double)M};
  bad = 0;
  // no term raised the reference: every value is -inf or lies below it (rows of a type's lowest value)
  odd |= M == kNoReference;
  if (!odd) {
#pragma unroll
    for (int w = 0; w < kSegWaves; ++w) t.sum += ldexp(sh.s[w], (int)fmaxf(sh.m[w] - M, -2000.f));
    return t;
  }
  __syncthreads();
  float m = x;
#pragma unroll 1
  for (int j = 0; j < kSegVecs; ++j) {
    float z[Seg::EPV];
    Seg::unpack(again(j), z);
#pragma unroll
    for (int e = 0; e < Seg::EPV; ++e) m = fmaxf(m, z[e]);
  }
  m = wave_max(m);
  if (lane == 0) sh.m[wave] = m;
  __syncthreads();
  for (int w = 0; w < kSegWaves; ++w) m = fmaxf(m, sh.m[w]);
  const float mr = m > -INFINITY ? m : 0.f;
  float S = exp_term(x, mr, c_hi, c_lo);
#pragma unroll 1
  for (int j = 0; j < kSegVecs; ++j) {
    float z[Seg::EPV];
    Seg::unpack(again(j), z);
#pragma unroll
    for (int e = 0; e < Seg::EPV; ++e) S += exp_term(z[e], mr, c_hi, c_lo);
  }
  const int wb = __ballot(!(S < INFINITY) || !(m < INFINITY)) != 0;
  const double s2 = wave_sum((double)S);
  if (lane == 0) {
    sh.s[wave] = s2;
    sh.odd[wave] = wb;
  }
  __syncthreads();
  for (int w = 0; w < kSegWaves; ++w) {
    t.sum += sh.s[w];
    bad |= sh.odd[w];
  }
  t.ref = (double)mr * ((double)c_hi + (double)c_lo);
  return t;
}

// Order-preserving 32-bit key of a float (larger float -> larger key).
__device__ __forceinline__ uint32_t order_key(float f) {
  const uint32_t u = __float_as_uint(f);
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7fffffffu) : ~k);
}
constexpr uint32_t kNegInfKey = 0x007fffffu;   // order_key(-inf)

// Host checks shared by the training entry points (defined in verify.hip).
bool shape_ok(int B, int G, int V, int dtype);
bool aligned16(const void* p);
inline bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 255u) == 0; }
inline size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace spec
