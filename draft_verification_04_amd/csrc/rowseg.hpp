// A logit row streamed by a workgroup (training kernels).
//
// A row's 16-byte body is cut into `nseg` segments, one workgroup each; a workgroup walks its segment in
// chunks of kSegThreads * kSegVecs vectors (64 KB), every thread holding kSegVecs of them in registers
// and issuing the next chunk's load as soon as it takes a vector.  The elements before the first and
// after the last whole vector (at most 7 + 7, rows that do not start or end on a 16-byte boundary)
// belong to segment 0, one per thread.
#pragma once

#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "common.hpp"
#include "spec_verify.h"

namespace spec {

constexpr int kSegThreads = 512;
constexpr int kSegWaves = kSegThreads / SPEC_WAVE;
// 16-byte vectors per thread: 32 registers; the kernels that read rows keep within 64 (8 waves per SIMD), the
// distillation gradient takes 66 (7)
constexpr int kSegVecs = 8;
constexpr int kSegWorkgroups = 512;   // a call's workgroups, at least, where rows are long enough
constexpr double kLog2eSeg = 1.44269504088896340736;

constexpr int kSegChunk = kSegThreads * kSegVecs;
constexpr int kMaxSegs = 16;
constexpr int kMaxSegVecs = 5 * kSegChunk;   // of a segment (its bitmap of listed tokens takes 20 KB)

// Segments of a row of V logits in a call of `rows` rows: two workgroups per CU at least, none shorter than a
// chunk.  One segment per row where there are rows enough: a workgroup's setup, and the joining of a row's
// segments, cost more than the idle CUs of a last round (lists of 256 on 672 rows of 129280 bf16: 84 us
// whole, 123 us in three segments).
inline int row_segments(int64_t rows, int V, int dtype) {
  const int vecs = V / (dtype == SPEC_BF16 ? 8 : 4);
  const int least = (vecs + kMaxSegVecs - 1) / kMaxSegVecs, most = (vecs + kSegChunk - 1) / kSegChunk;
  const int64_t want = (kSegWorkgroups + rows - 1) / rows;
  int n = want > most ? most : (int)want;
  if (n < least) n = least;
  return n < 1 ? 1 : n;   // at most kMaxSegs: V <= SPEC_MAX_V (fp32: half)
}

// Which row (request i, position k) unit o of a call is; false: none.  With lengths the units are the live
// rows (k < L_i, a valid temperature) in order, found by a prefix sum over the requests, so that the
// workgroups without a row come last and exit together: between the live ones they held slots that rows
// wait for (256 x 16 rows, half of them live: 190 us in place, 142 us this way).  Beyond kLiveRequests
// requests every workgroup would sum too many lengths, and the rows stay in place.
constexpr int kLivePer = 8, kLiveRequests = kSegThreads * kLivePer;

struct LiveShared {
  int wave[kSegWaves];
  int i, k;
};

__device__ __forceinline__ bool live_row(LiveShared& sh, int o, int B, int G, const int32_t* lengths,
                                         const float* temperature, int& i, int& k) {
  auto live = [&](int q) -> int {
    const int L = lengths ? lengths[q] : G;
    const float T = temperature[q];
    return L <= G && T > 0.f && T < INFINITY ? L : 0;
  };
  if (!lengths || B > kLiveRequests) {
    i = o / G;
    k = o - i * G;
    return k < live(i);
  }
  const int tid = (int)threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int per = (B + kSegThreads - 1) / kSegThreads;
  int n[kLivePer], sum = 0;
#pragma unroll
  for (int u = 0; u < kLivePer; ++u) {
    n[u] = 0;
    if (u < per && tid * per + u < B) n[u] = max(live(tid * per + u), 0);
    sum += n[u];
  }
  const int in = wave_inclusive_scan(sum);
  if (lane == 63) sh.wave[wave] = in;
  if (tid == 0) sh.i = -1;
  lds_barrier();
  int before = in - sum;
#pragma unroll
  for (int w = 0; w < kSegWaves; ++w) before += w < wave ? sh.wave[w] : 0;
  if (o >= before && o < before + sum) {
    int at = o - before;
#pragma unroll
    for (int u = 0; u < kLivePer; ++u) {
      if (at >= 0 && at < n[u]) {
        sh.i = tid * per + u;
        sh.k = at;
      }
      at -= n[u];
    }
  }
  lds_barrier();
  i = __builtin_amdgcn_readfirstlane(sh.i);
  k = __builtin_amdgcn_readfirstlane(sh.k);
  return i >= 0;
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
  // the thread's vectors of the first chunk; loads issued together, clamped to the last vector (-inf when
  // the segment has none)
  __device__ __forceinline__ void load(const char* row, uint4 (&d)[kSegVecs]) const {
    const uint4* vp = reinterpret_cast<const uint4*>(row + (size_t)head * ES);
    if (vb < ve) {
#pragma unroll
      for (int j = 0; j < kSegVecs; ++j) d[j] = load_nt(vp + min(vb + j * kSegThreads + (int)threadIdx.x, ve - 1));
    } else {
#pragma unroll
      for (int j = 0; j < kSegVecs; ++j) d[j] = make_uint4(kNegInf, kNegInf, kNegInf, kNegInf);
    }
  }
  // take(v, x) for every vector v of the chunk at c that the thread holds, x its 16 bytes (-inf past the
  // end); each register is refilled with the next chunk's vector.  The loads stand outside of every
  // branch (clamped past the end): a load that only some paths issue makes each wait one for every load
  // in flight
  template <class Take>
  __device__ __forceinline__ void walk_chunk(const char* row, int c, uint4 (&d)[kSegVecs], Take take) const {
    const uint4* vp = reinterpret_cast<const uint4*>(row + (size_t)head * ES);
#pragma unroll
    for (int j = 0; j < kSegVecs; ++j) {
      const int v = c + j * kSegThreads + (int)threadIdx.x;
      if (c + j * kSegThreads < ve) {
        uint4 x = d[j];
        if (c + (j + 1) * kSegThreads > ve && v >= ve) x = make_uint4(kNegInf, kNegInf, kNegInf, kNegInf);
        take(v, x);
      }
      d[j] = load_nt(vp + min(v + kSegChunk, ve - 1));
    }
  }
  template <class Take>
  __device__ __forceinline__ void walk(const char* row, uint4 (&d)[kSegVecs], Take take) const {
#pragma unroll 1
    for (int c = vb; c < ve; c += kSegChunk) walk_chunk(row, c, d, take);
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

// log2(e) / T, finite in fp32 for every T > 0 (T towards 0 is the argmax); and as a float pair, c_hi toward
// zero and c_lo > 0 (so that a logit of -inf gives an exponent of -inf, never NaN).
__device__ __forceinline__ double scale_of(float T) { return fmin(kLog2eSeg / (double)T, 3.4028234663852886e38); }

__device__ __forceinline__ void split_scale(float T, float& c_hi, float& c_lo) {
  const double c = scale_of(T);
  c_hi = __double2float_rz(c);
  c_lo = fmaxf((float)(c - (double)c_hi), 1.4e-45f);
}

// Added in pairs: log2 N roundings of a term.
template <int N>
__device__ __forceinline__ float pair_sum(float (&e)[N]) {
#pragma unroll
  for (int w = 1; w < N; w <<= 1)
#pragma unroll
    for (int j = 0; j + w < N; j += 2 * w) e[j] += e[j + w];
  return e[0];
}

// Sum of exp2(z c_f - M) over a vector, c_f = log2(e) / T rounded to fp32: one multiply-add per term.  M is
// an integer, the same for the whole segment: the ceiling of the largest exponent of its first chunk
// (pick_reference, which keeps that largest logit m).  With u = 2^-24, the sum is off by (relative)
//  - the rounding of c_f, which shifts every exponent by z (c - c_f): the shift of the logit whose exponent is the
//    sum's own, M + log2(sum), is common to the segment and goes into its reference in fp64 (segment_sum); what is
//    left is at most u |x| per term, x its distance from there in nats, and over a softmax of V terms
//    E|x| <= ln V + 1.4;
//  - the rounding of each exponent, half a step: below 2^6 in size 2^-19, 22 u of its term, and terms further
//    below have no weight beside the largest.  A later value may stand 2^63 above M before a thread's sum says
//    so (one of 43 T nats more than the largest of 32768): past that the exponents' rounding would grow to 2^-18,
//    44 u, and the segment is summed again by exp_term in segment_sum.  So is one whose first chunk has no
//    value, one with NaN or +inf and one with exponents past 2^22 (an fp32 reference no longer tells their
//    neighbours apart);
//  - an ulp of exp2 (2 u) and 44 roundings of a thread's sum: together below 110 u for every V.
template <int N>
__device__ __forceinline__ float exp_sum(const float (&z)[N], float c_f, float M) {
  float e[N];
#pragma unroll
  for (int j = 0; j < N; ++j) e[j] = __builtin_amdgcn_exp2f(fmaf(z[j], c_f, -M));
  return pair_sum(e);
}

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

// Scratch of pick_reference and segment_sum.
struct SegSumShared {
  double s[kSegWaves];
  float m[kSegWaves];
  int odd[kSegWaves];
};

// A segment's scale and reference (see exp_sum).
struct Reference {
  double c;      // log2(e) / T
  float c_f, M;
  double ref;    // M and the shift of m by c_f's rounding: the sum is S * 2^ref
  bool ok;       // false: there is no reference
};

// From the workgroup's threads' largest values.
__device__ __forceinline__ Reference pick_reference(SegSumShared& sh, float zm, float T) {
  const int wave = (int)threadIdx.x >> 6, lane = (int)threadIdx.x & 63;
  zm = wave_max(zm);
  if (lane == 0) sh.m[wave] = zm;
  lds_barrier();
#pragma unroll
  for (int w = 0; w < kSegWaves; ++w) zm = fmaxf(zm, sh.m[w]);
  Reference r;
  r.c = scale_of(T);
  r.c_f = (float)r.c;
  r.M = ceilf(zm * r.c_f);
  r.ok = fabsf(r.M) < 0x1p22f;
  if (!r.ok) r.M = 0.f;
  r.ref = (double)r.M + (r.ok ? (double)zm * (r.c - (double)r.c_f) : 0.0);
  return r;
}

// The workgroup's sum (and whether a NaN or +inf was among the values) from its threads' sums S1; every
// thread gets the result.  again(v) reads body vector v once more and x is the thread's scalar: used
// only when a sum left the range, or without a reference.
template <bool BF16, class Again>
__device__ __forceinline__ SegSum segment_sum(SegSumShared& sh, float S1, const Reference& rf, float T,
                                              const RowSeg<BF16>& g, Again again, float x, int& bad) {
  using Seg = RowSeg<BF16>;
  const int wave = (int)threadIdx.x >> 6, lane = (int)threadIdx.x & 63;
  const double ws = wave_sum((double)S1);
  const int wo = __ballot(!(S1 <= 0x1p63f)) != 0;
  if (lane == 0) {
    sh.s[wave] = ws;
    sh.odd[wave] = wo;
  }
  __syncthreads();
  SegSum t{0.0, rf.ref};
  int odd = !rf.ok;
#pragma unroll
  for (int w = 0; w < kSegWaves; ++w) {
    t.sum += sh.s[w];
    odd |= sh.odd[w];
  }
  bad = 0;
  if (!odd) {
    // from m's shift to that of the sum's own exponent, log2(sum) / c further (1 <= 2 sum)
    t.ref += (double)ilogb(t.sum) * (1.0 - (double)rf.c_f / rf.c);
    return t;
  }
  t.sum = 0.0;
  float c_hi, c_lo;
  split_scale(T, c_hi, c_lo);
  __syncthreads();
  float m = x;
#pragma unroll 1
  for (int v = g.vb + (int)threadIdx.x; v < g.ve; v += kSegThreads) {
    float z[Seg::EPV];
    Seg::unpack(again(v), z);
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
  for (int v = g.vb + (int)threadIdx.x; v < g.ve; v += kSegThreads) {
    float z[Seg::EPV];
    Seg::unpack(again(v), z);
#pragma unroll
    for (int e = 0; e < Seg::EPV; ++e) z[e] = exp_term(z[e], mr, c_hi, c_lo);
    S += pair_sum(z);
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
  t.ref = (double)mr * rf.c;   // exactly the exponent of a logit mr, also where mr c is so large that its neighbours differ by more
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
inline bool overlap(const void* a, size_t an, const void* b, size_t bn) {   // NULL overlaps nothing
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + bn && y < x + an;
}
inline size_t round256(size_t x) { return (x + 255) & ~(size_t)255; }

}  // namespace spec
