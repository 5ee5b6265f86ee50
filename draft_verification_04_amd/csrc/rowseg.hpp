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

// exp2((z - m) c): the difference to the reference first, so that its size, not the logit's, sets
// the rounding (at most about 2^-24 |z - m| c relative, weighed by e^-|z - m|/T).
__device__ __forceinline__ float exp_term(float z, float m, float c_hi, float c_lo) {
  const float dz = z - m;
  return __builtin_amdgcn_exp2f(fmaf(dz, c_lo, dz * c_hi));
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
