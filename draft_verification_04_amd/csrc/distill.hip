// Distillation of the draft distribution from a teacher's top logits on gfx950, with its gradient.
//
// For a draft row z, q = softmax(z / T) over the whole row, a teacher list S of tokens with
// probabilities p_e (renormalised over the list, or scaled by the teacher's own normaliser, the rest
// r_t kept as one bucket against the draft's mass r_s outside the list):
//   KL: sum_e p_e ln(p_e / q_e) + r_t ln(r_t / r_s)
//   TV: sum_e max(p_e - q_e, 0) + max(r_t - r_s, 0)   (DSpark paper, §3.3 and Eq. 8)
// Their derivatives are multiples of q outside the list and q b - c_e in it:
//   KL: b = sum of p_e + r_t (1, unless the teacher's normaliser is rounded or lies below its list's),
//       a = b - r_t / r_s, c_e = p_e
//   TV: b = sum of q_e over p_e > q_e, + r_s if r_t > r_s;  a = b - [r_t > r_s];  c_e = [p_e > q_e] q_e
//   dz_v = grad_loss / T * (q_v a, or q_e b - c_e)
//
// r_s is summed over the tokens outside the list, never taken as 1 - sum of q_e: where the list holds
// nearly all of q the difference has no correct digit, and a and ln r_s hang on it.
//
// The work is one read of the rows (forward) and one read and one write (backward):
//   distill_stream_kernel -- one workgroup per row (or segment, when there are few rows): marks the
//       listed tokens in an LDS bitmap (a byte per 16-byte vector of bf16, so a vector without a listed
//       token costs one LDS byte), takes them out and sums exp of the rest; then, when the row is
//       whole, its first wave forms the list's terms in fp64 (finish_row).
//   distill_finish_kernel -- the same last step over a row's segments.
//   distill_status_kernel -- one wave per request: the rows' findings, and NaN for a failed request.
//   distill_grad_kernel -- one workgroup per (row, segment): q a of every token as (q / r_s) (a r_s),
//       then, behind a barrier, the listed tokens' own values over it.
// MI355X: 512 x 7 rows of 151936 bf16, half of them live: forward 109-116 us (4.7-5.0 TB/s), backward 291-317
// (5.2-5.6 TB/s read and written; a copy: 4.9); 2048 rows of 129280, all live, K = 200, with the tail: 89 us
// (6.0 TB/s).
#include "common.hpp"
#include "rowseg.hpp"
#include "spec_verify.h"

namespace spec {
namespace {

constexpr double kLn2Seg = 0.69314718055994530942;
constexpr int kFlagBad = 1;    // NaN or +inf outside the list
constexpr int kFlagTwice = 2;  // a token id named twice

struct DistillSeg {
  double sum, ref;   // sum of exp(z / T) over the segment's tokens outside the list: sum * 2^ref
  int32_t flags, pad;
};

struct DistillArgs {
  int B, G, V, K, nseg, mode;
  const void* draft;
  const int32_t* ids;
  const float* values;
  const float* teacher_lse;
  const int32_t* lengths;
  const float* temperature;
  float* loss;
  double* saved;
  int32_t* status;
  DistillSeg* segs;        // [B * G, nseg]
  int32_t* row_status;     // [B * G]
  const float* grad_loss;  // backward
  void* grad;
};

// A used entry names a token and has a logit above -inf (a NaN logit is used, and bad).
__device__ __forceinline__ bool used_entry(int id, float v) { return id != -1 && !(v == -INFINITY); }

__device__ __forceinline__ double wave_max_d(double x) {
  return wave_reduce(x, [](double p, double q) { return fmax(p, q); });
}

// A row's list beside its draft logits, for finish_row.
struct ListShared {
  int32_t id[SPEC_MAX_TEACHER_K];
  float val[SPEC_MAX_TEACHER_K], z[SPEC_MAX_TEACHER_K];
  double el[SPEC_MAX_TEACHER_K], te[SPEC_MAX_TEACHER_K];
};

// The last step of a row, by one wave: the list (K entries, z the draft's logits at the tokens) and, in lanes
// s < nseg, the sums seg * 2^ref of exp(z / T) outside the list (0 in the other lanes).  All in powers of
// two.  One wave, not the row's eight: the fp64 reductions cost a wave the same whatever it holds, and they
// were a quarter of the whole call by eight.  exp2 and log2 stand in few places (the code runs once per
// row and is cold then); log2 takes its four arguments from four lanes.
__device__ __forceinline__ void finish_row(ListShared& sh, const DistillArgs& a, size_t r, double seg, double ref, int rst,
                                           float T) {
  const int lane = (int)threadIdx.x & 63, K = a.K;
  const double c = scale_of(T);
  const bool tail = a.teacher_lse != nullptr;
  const float tl = tail ? a.teacher_lse[r] : 0.f;
  float vmax = -INFINITY, dmax = -INFINITY;
  int nused = 0;
#pragma unroll 1
  for (int e0 = 0; e0 < K; e0 += SPEC_WAVE) {
    const int e = e0 + lane;
    bool used = false;
    if (e < K) {
      const int id = sh.id[e];
      const float v = sh.val[e], z = sh.z[e];
      used = used_entry(id, v);
      if (used) {
        if (id < 0 || id >= a.V) {
          rst |= SPEC_REQ_BAD_TOKEN;
        } else {
          if (!(v < INFINITY) || !(z < INFINITY)) rst |= SPEC_REQ_NONFINITE;
          vmax = fmaxf(vmax, v);
          dmax = fmaxf(dmax, z);
        }
      }
    }
    nused += (int)__popcll(__ballot(used));
  }
  const bool seg_on = seg > 0.0;
  const double mo = wave_max_d(seg_on ? ref : -INFINITY);   // the largest reference outside the list
  const bool outside = mo > -INFINITY;
  const double tmax = (double)wave_max(vmax) * c, zmax = fmax((double)wave_max(dmax) * c, mo);
  if (tail && !(fabsf(tl) < INFINITY)) rst |= SPEC_REQ_NONFINITE;
  if (!(zmax > -INFINITY)) rst |= SPEC_REQ_NONFINITE;
  rst = wave_or_i(rst);
  double* sv = a.saved + r * SPEC_DISTILL_SAVED;
  if (nused == 0 || rst != 0) {   // no entry: the row is not read
    if (lane == 0) {
      a.loss[r] = nused == 0 ? 0.f : NAN;
      sv[0] = NAN;
      a.row_status[r] = nused == 0 ? 0 : rst;
    }
    return;
  }
  double lsum = 0.0, tsum = 0.0;
#pragma unroll 1
  for (int e0 = 0; e0 < K; e0 += SPEC_WAVE) {
    const int e = e0 + lane;
    double x = -INFINITY, y = -INFINITY;
    if (e < K && used_entry(sh.id[e], sh.val[e])) {
      x = (double)sh.z[e] * c - zmax;
      y = (double)sh.val[e] * c - tmax;
    }
    x = exp2(x);
    y = exp2(y);
    if (e < K) {
      sh.el[e] = x;
      sh.te[e] = y;
    }
    lsum += x;
    tsum += y;
  }
  lsum = wave_sum(lsum);
  tsum = wave_sum(tsum);
  // lanes s the segments' shares exp2(ref - mo), lane 62 exp2(tmax - t), lane 63 exp2(mo - zmax)
  static_assert(kMaxSegs <= 62, "lanes of the segments");
  const double t = tail ? (double)tl * kLog2eSeg : tmax;   // p = exp2((v c - t) - tl2)
  const double sc = exp2(lane == 62 ? tmax - t : lane == 63 ? mo - zmax : ref - mo);
  const double out = wave_sum(seg_on ? seg * sc : 0.0);
  const double rest = outside ? out * read_lane(sc, 63) : 0.0;   // outside the list, against zmax
  const double tot = rest + lsum, itot = 1.0 / tot;
  const double ps = tail ? read_lane(sc, 62) : 1.0 / tsum;
  const double rt = (tail && nused < a.V) ? fmax(0.0, 1.0 - tsum * ps) : 0.0;
  const double rs = rest * itot;
  const int which = lane & 3;
  const double lg = log2(which == 0 ? out : which == 1 ? tot : which == 2 ? tsum : rt);
  const double lout = read_lane(lg, 0), lt = read_lane(lg, 1), lrt = read_lane(lg, 3);
  // (the normalisers stay in two parts: beside logits of 1e17 T and more their logarithm would be lost)
  const double tl2 = tail ? 0.0 : read_lane(lg, 2);
  double loss = 0.0, bv = 0.0;
#pragma unroll 1
  for (int e = lane; e < K; e += SPEC_WAVE) {
    const double pe = sh.te[e] * ps, qe = sh.el[e] * itot;
    if (a.mode == SPEC_DISTILL_KL) {
      if (pe > 0.0) loss += pe * (((double)sh.val[e] * c - t - tl2) - ((double)sh.z[e] * c - zmax - lt));
    } else if (pe > qe) {
      loss += pe - qe;
      bv += qe;
    }
  }
  loss = wave_sum(loss);
  double ars;   // a r_s: q a = (q / r_s) (a r_s) outside the list, finite however small r_s
  if (a.mode == SPEC_DISTILL_KL) {
    bv = tail ? tsum * ps + rt : 1.0;
    ars = bv * rs - rt;
    // in logs (the tail may lie hundreds of nats below the list); +inf when the draft leaves no mass there
    if (rt > 0.0) loss += rt * (lrt - (outside ? mo - zmax + lout - lt : -INFINITY));
    loss *= kLn2Seg;
  } else {
    bv = wave_sum(bv);
    const bool up = rt > rs;
    if (up) {
      loss += rt - rs;
      bv += rs;
    }
    ars = (bv - (up ? 1.0 : 0.0)) * rs;
  }
  if (lane != 0) return;
  // q / r_s = exp2((z - m) c - sv[1]): the logit nearest the largest exponent as reference
  const float m = outside ? (float)(mo / c) : 0.f;
  sv[0] = (double)m;
  sv[1] = outside ? mo - (double)m * c + lout : 0.0;
  sv[2] = outside ? ars : 0.0;
  sv[3] = bv;
  sv[4] = t;
  sv[5] = tl2;
  sv[6] = zmax;
  sv[7] = lt;
  a.loss[r] = (float)loss;
  a.row_status[r] = 0;
}

__device__ __forceinline__ int row_flags(int f) {
  return (f & kFlagBad ? SPEC_REQ_NONFINITE : 0) | (f & kFlagTwice ? SPEC_REQ_BAD_LIST : 0);
}

template <bool BF16>
__global__ __launch_bounds__(kSegThreads) __attribute__((amdgpu_waves_per_eu(8)))
void distill_stream_kernel(DistillArgs a) {
  using Seg = RowSeg<BF16>;
  constexpr int EPV = Seg::EPV;
  extern __shared__ __attribute__((aligned(16))) uint32_t bits[];   // listed tokens of the segment
  __shared__ uint32_t xbits;
  __shared__ SegSumShared ss;
  __shared__ ListShared ls;
  __shared__ int sflags;
  __shared__ LiveShared live;
  const int o = (int)(blockIdx.x / (unsigned)a.nseg), seg = (int)(blockIdx.x - (unsigned)o * a.nseg);
  int i, k;
  if (!live_row(live, o, a.B, a.G, a.lengths, a.temperature, i, k)) return;   // the status kernel fills the other rows
  const int r = i * a.G + k;
  const float T = a.temperature[i];
  const int tid = threadIdx.x;
  const int e0 = min(tid, a.K - 1);
  const int id = a.ids[(size_t)r * a.K + e0];
  const float val = a.values[(size_t)r * a.K + e0];
  const char* row = reinterpret_cast<const char*>(a.draft) + (size_t)r * (size_t)a.V * Seg::ES;
  const Seg g(row, a.V, seg, a.nseg);
  uint4 d[kSegVecs];
  float x = g.load_scalar(row);
  g.load(row, d);
  const int words = ((g.ve - g.vb) * EPV + 127) / 128;   // 16 bytes each
  for (int w = tid; w < words; w += kSegThreads) reinterpret_cast<uint4*>(bits)[w] = make_uint4(0, 0, 0, 0);
  if (tid == 0) xbits = sflags = 0;
  lds_barrier();
  const bool listed = tid < a.K && used_entry(id, val) && id >= 0 && id < a.V;
  if (tid < a.K && a.nseg == 1) {
    ls.id[tid] = id;
    ls.val[tid] = val;
    ls.z[tid] = load_elem<BF16>(row, listed ? id : 0);
  }
  if (listed) {
    const int body = id - g.head, rel = body - g.vb * EPV;
    if (id < g.head || id >= g.tail0) {
      if (seg == 0) {
        const uint32_t bit = 1u << (id < g.head ? id : g.head + (id - g.tail0));
        if (atomicOr(&xbits, bit) & bit) atomicOr(&sflags, kFlagTwice);
      }
    } else if (rel >= 0 && body < g.ve * EPV) {
      const uint32_t bit = 1u << (rel & 31);
      if (atomicOr(&bits[rel >> 5], bit) & bit) atomicOr(&sflags, kFlagTwice);
    }
  }
  lds_barrier();
  if (tid < g.nx && ((xbits >> tid) & 1u)) x = -INFINITY;
  const uint8_t* bytes = reinterpret_cast<const uint8_t*>(bits);
  // vector v (in the body) without its listed tokens
  auto unlisted = [&](uint4 q, int v) -> uint4 {
    const int lv = v - g.vb;
    uint32_t w;
    if constexpr (BF16) w = bytes[lv];
    else w = (bytes[lv >> 1] >> ((lv & 1) * 4)) & 15u;
    if (w) {
      uint32_t p[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        uint32_t m;   // ones over the listed values of the word
        if constexpr (BF16)
          m = ((uint32_t)__builtin_amdgcn_sbfe((int)w, 2 * h, 1) & 0xffffu) |
              ((uint32_t)__builtin_amdgcn_sbfe((int)w, 2 * h + 1, 1) & 0xffff0000u);
        else
          m = (uint32_t)__builtin_amdgcn_sbfe((int)w, h, 1);
        p[h] = (p[h] & ~m) | (Seg::kNegInf & m);
      }
      q = make_uint4(p[0], p[1], p[2], p[3]);
    }
    return q;
  };
  float zm = x;
#pragma unroll
  for (int j = 0; j < kSegVecs; ++j) {
    const int v = g.vb + j * kSegThreads + tid;
    if (v - tid < g.ve) {
      float z[EPV];
      Seg::unpack(unlisted(d[j], min(v, g.ve - 1)), z);
#pragma unroll
      for (int e = 0; e < EPV; ++e) zm = fmaxf(zm, z[e]);   // past the end: the last vector again
    }
    asm volatile("" : "+v"(zm));
  }
  forget(d);
  const Reference rf = pick_reference(ss, zm, T);
  float S = 0.f;
  g.walk(row, d, [&](int v, const uint4& q) {
    float z[EPV];
    Seg::unpack(unlisted(q, min(v, g.ve - 1)), z);
    S += exp_sum<EPV>(z, rf.c_f, rf.M);
    asm volatile("" : "+v"(S));   // one vector's values at a time: registers
  });
  if (g.nx > 0) {
    const float z1[1] = {x};
    S += exp_sum<1>(z1, rf.c_f, rf.M);
  }
  int bad;
  const SegSum t = segment_sum<BF16>(
      ss, S, rf, T, g,
      [&](int v) { return unlisted(reinterpret_cast<const uint4*>(row + (size_t)g.head * Seg::ES)[v], v); }, x, bad);
  const int flags = sflags | (bad ? kFlagBad : 0);
  if (a.nseg == 1) {
    if (tid < SPEC_WAVE) finish_row(ls, a, (size_t)r, tid == 0 ? t.sum : 0.0, t.ref, row_flags(flags), T);
  } else if (tid == 0) {
    a.segs[(size_t)r * a.nseg + seg] = DistillSeg{t.sum, t.ref, flags, 0};
  }
}

// One wave per row of several segments.
constexpr int kFinishWaves = 4;

template <bool BF16>
__global__ __launch_bounds__(kFinishWaves * SPEC_WAVE) void distill_finish_kernel(DistillArgs a) {
  __shared__ ListShared ls[kFinishWaves];
  const int wave = (int)threadIdx.x >> 6, lane = (int)threadIdx.x & 63;
  const int64_t r = (int64_t)blockIdx.x * kFinishWaves + wave;
  if (r >= (int64_t)a.B * a.G) return;
  const int i = (int)(r / a.G), k = (int)(r - (int64_t)i * a.G);
  const int L = a.lengths ? a.lengths[i] : a.G;
  const float T = a.temperature[i];
  if (k >= L || L > a.G || !(T > 0.f && T < INFINITY)) return;
  const DistillSeg mine = a.segs[(size_t)r * a.nseg + min(lane, a.nseg - 1)];
  const bool on = lane < a.nseg;
  const char* row = reinterpret_cast<const char*>(a.draft) + (size_t)r * (size_t)a.V * RowSeg<BF16>::ES;
  int id[SPEC_MAX_TEACHER_K / SPEC_WAVE];
  float val[SPEC_MAX_TEACHER_K / SPEC_WAVE];
#pragma unroll
  for (int u = 0; u < SPEC_MAX_TEACHER_K / SPEC_WAVE; ++u) {
    const size_t e = (size_t)r * a.K + min(lane + u * SPEC_WAVE, a.K - 1);
    id[u] = a.ids[e];
    val[u] = a.values[e];
  }
#pragma unroll
  for (int u = 0; u < SPEC_MAX_TEACHER_K / SPEC_WAVE; ++u) {
    const float z = load_elem<BF16>(row, id[u] >= 0 && id[u] < a.V ? id[u] : 0);
    if (lane + u * SPEC_WAVE < a.K) {
      ls[wave].id[lane + u * SPEC_WAVE] = id[u];
      ls[wave].val[lane + u * SPEC_WAVE] = val[u];
      ls[wave].z[lane + u * SPEC_WAVE] = z;
    }
  }
  finish_row(ls[wave], a, (size_t)r, on ? mine.sum : 0.0, mine.ref, row_flags(on ? mine.flags : 0), T);
}

// One wave per request.
__global__ __launch_bounds__(256) void distill_status_kernel(DistillArgs a) {
  const int i = (int)blockIdx.x * 4 + ((int)threadIdx.x >> 6), k = (int)threadIdx.x & 63;
  if (i >= a.B) return;
  const int L = a.lengths ? a.lengths[i] : a.G;
  const float T = a.temperature[i];
  const size_t r = (size_t)i * a.G + min(k, a.G - 1);
  int st = 0;
  if (L < 0 || L > a.G) st = SPEC_REQ_BAD_LENGTH;
  else if (!(T > 0.f && T < INFINITY)) st = SPEC_REQ_BAD_TEMPERATURE;
  else st = wave_or_i(k < L ? a.row_status[r] : 0);
  if (k == 0 && a.status) a.status[i] = st;
  if (k < a.G && (st != 0 || k >= L)) {   // a failed request, or a row that is not read
    a.loss[r] = st != 0 ? NAN : 0.f;
    a.saved[r * SPEC_DISTILL_SAVED] = NAN;
  }
}

// Workgroup barrier behind which every load and store issued before it is complete.
__device__ __forceinline__ void memory_barrier() {
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// fp32 -> bf16 pair, round to nearest, ties to even.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  bf16x2 v;
  v.x = (__bf16)lo;
  v.y = (__bf16)hi;
  return __builtin_bit_cast(uint32_t, v);
}

template <bool BF16>
__device__ __forceinline__ void store_elem(char* row, int id, float g) {
  if constexpr (BF16) reinterpret_cast<__bf16*>(row)[id] = (__bf16)g;
  else reinterpret_cast<float*>(row)[id] = g;
}

template <bool BF16>
__global__ __launch_bounds__(kSegThreads) void distill_grad_kernel(DistillArgs a) {
  using Seg = RowSeg<BF16>;
  constexpr int EPV = Seg::EPV;
  const int r = (int)(blockIdx.x / (unsigned)a.nseg), seg = (int)(blockIdx.x - (unsigned)r * a.nseg);
  const int i = r / a.G;
  const int tid = threadIdx.x;
  const double* sv = a.saved + (size_t)r * SPEC_DISTILL_SAVED;
  const double md = sv[0];
  const char* row = reinterpret_cast<const char*>(a.draft) + (size_t)r * (size_t)a.V * Seg::ES;
  char* out = reinterpret_cast<char*>(a.grad) + (size_t)r * (size_t)a.V * Seg::ES;
  const Seg g(row, a.V, seg, a.nseg);
  uint4* ov = reinterpret_cast<uint4*>(out + (size_t)g.head * Seg::ES);
  if (!(md == md)) {   // a row with no loss
#pragma unroll
    for (int j = 0; j < kSegVecs; ++j) {
      const int v = g.vb + j * kSegThreads + tid;
      if (v < g.ve) ov[v] = make_uint4(0, 0, 0, 0);
    }
    if (tid < g.nx) store_elem<BF16>(out, g.id_of_scalar(tid), 0.f);
    return;
  }
  // the thread's list entry, when its token lies in this segment
  const float T = a.temperature[i];
  const double s = (double)a.grad_loss[r] / (double)T;
  int id = -1;
  float val = -INFINITY, ze = 0.f;
  if (tid < a.K) {
    id = a.ids[(size_t)r * a.K + tid];
    val = a.values[(size_t)r * a.K + tid];
    const int body = id - g.head;
    const bool mine = (id < g.head || id >= g.tail0) ? seg == 0 : (body >= g.vb * EPV && body < g.ve * EPV);
    if (!used_entry(id, val) || id < 0 || id >= a.V || !mine) id = -1;
    if (id >= 0) ze = load_elem<BF16>(row, id);
  }
  uint4 d[kSegVecs];
  g.load(row, d);
  const float x = g.load_scalar(row);
  float c_hi, c_lo;
  split_scale(T, c_hi, c_lo);
  const float m = (float)md, l2 = (float)sv[1];
  // the factor past fp32's range (grad_loss / T of 2^127 and more) is multiplied in two steps: as inf it would
  // make the tokens without mass NaN
  const double fd = s * sv[2];
  const int up = fabs(fd) < INFINITY ? max(ilogb(fd) - 126, 0) : 0;
  const float f = (float)ldexp(fd, -up);
  // every load of the segment is done in every wave before the first store (grad may be draft)
  memory_barrier();
  auto grad_of = [&](float z) {
    const float dz = z - m;   // q / r_s of a token outside the list
    return ldexpf(f * __builtin_amdgcn_exp2f(fmaf(dz, c_lo, fmaf(dz, c_hi, -l2))), up);
  };
#pragma unroll
  for (int j = 0; j < kSegVecs; ++j) {
    const int v = g.vb + j * kSegThreads + tid;
    float z[EPV];
    Seg::unpack(d[j], z);
    uint4 o;
    if constexpr (BF16) {
      o = make_uint4(pack_bf16(grad_of(z[0]), grad_of(z[1])), pack_bf16(grad_of(z[2]), grad_of(z[3])),
                     pack_bf16(grad_of(z[4]), grad_of(z[5])), pack_bf16(grad_of(z[6]), grad_of(z[7])));
    } else {
      o = make_uint4(__float_as_uint(grad_of(z[0])), __float_as_uint(grad_of(z[1])),
                     __float_as_uint(grad_of(z[2])), __float_as_uint(grad_of(z[3])));
    }
    if (v < g.ve) ov[v] = o;
  }
  if (tid < g.nx) store_elem<BF16>(out, g.id_of_scalar(tid), grad_of(x));
  memory_barrier();   // the segment's stores are done: the listed tokens' go over them
  if (id >= 0) {
    const double c2 = scale_of(T);
    const double q = exp2((double)ze * c2 - sv[6] - sv[7]), p = exp2((double)val * c2 - sv[4] - sv[5]);
    const double c = a.mode == SPEC_DISTILL_KL ? p : (p > q ? q : 0.0);
    store_elem<BF16>(out, id, (float)(s * (q * sv[3] - c)));
  }
}

bool list_ok(int B, int G, int V, int dtype, int K) {
  return shape_ok(B, G, V, dtype) && K >= 1 && K <= SPEC_MAX_TEACHER_K;
}

}  // namespace
}  // namespace spec

using namespace spec;

extern "C" size_t spec_distill_workspace_size(int32_t B, int32_t gamma, int32_t V, int32_t K) {
  if (!list_ok(B, gamma, V, SPEC_BF16, K)) return 0;
  const size_t rows = (size_t)B * gamma;
  return round256(rows * kMaxSegs * sizeof(DistillSeg)) + round256(rows * sizeof(int32_t));
}

extern "C" int32_t spec_distill_loss(int32_t B, int32_t gamma, int32_t V, int32_t dtype, const void* draft_logits,
                                     int32_t K, const int32_t* teacher_ids, const float* teacher_values,
                                     const float* teacher_lse, int32_t mode, const int32_t* lengths,
                                     const float* temperature, float* loss_out, double* saved_out, int32_t* status,
                                     void* workspace, size_t workspace_bytes, void* stream) {
  if (!list_ok(B, gamma, V, dtype, K)) return SPEC_ERR_INVALID_ARG;
  if (mode != SPEC_DISTILL_KL && mode != SPEC_DISTILL_TV) return SPEC_ERR_INVALID_ARG;
  if (!draft_logits || !teacher_ids || !teacher_values || !temperature || !loss_out || !saved_out)
    return SPEC_ERR_INVALID_ARG;
  if (!aligned16(draft_logits)) return SPEC_ERR_INVALID_ARG;
  if (!workspace || !aligned256(workspace) || workspace_bytes < spec_distill_workspace_size(B, gamma, V, K))
    return SPEC_ERR_WORKSPACE;
  DistillArgs a{};
  a.B = B; a.G = gamma; a.V = V; a.K = K; a.mode = mode;
  const uint64_t rows = (uint64_t)B * gamma;
  a.nseg = row_segments((int64_t)rows, V, dtype);
  if (rows * a.nseg * kSegThreads > 0xffffffffull) return SPEC_ERR_UNSUPPORTED;
  a.draft = draft_logits; a.ids = teacher_ids; a.values = teacher_values; a.teacher_lse = teacher_lse;
  a.lengths = lengths; a.temperature = temperature; a.loss = loss_out; a.saved = saved_out; a.status = status;
  a.segs = reinterpret_cast<DistillSeg*>(workspace);
  a.row_status = reinterpret_cast<int32_t*>(reinterpret_cast<char*>(workspace) +
                                            round256(rows * kMaxSegs * sizeof(DistillSeg)));
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const dim3 grid((unsigned)(rows * a.nseg));
  const int elems = dtype == SPEC_BF16 ? 8 : 4, vecs = (V / elems + a.nseg - 1) / a.nseg;
  const unsigned lds = (unsigned)((vecs * elems + 127) / 128 * 16 + 16);
  if (dtype == SPEC_BF16) {
    hipLaunchKernelGGL(distill_stream_kernel<true>, grid, dim3(kSegThreads), lds, s, a);
    if (a.nseg > 1)
      hipLaunchKernelGGL(distill_finish_kernel<true>, dim3((unsigned)((rows + kFinishWaves - 1) / kFinishWaves)),
                         dim3(kFinishWaves * SPEC_WAVE), 0, s, a);
  } else {
    hipLaunchKernelGGL(distill_stream_kernel<false>, grid, dim3(kSegThreads), lds, s, a);
    if (a.nseg > 1)
      hipLaunchKernelGGL(distill_finish_kernel<false>, dim3((unsigned)((rows + kFinishWaves - 1) / kFinishWaves)),
                         dim3(kFinishWaves * SPEC_WAVE), 0, s, a);
  }
  hipLaunchKernelGGL(distill_status_kernel, dim3((unsigned)(B + 3) / 4), dim3(256), 0, s, a);
  return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_ERR_HIP;
}

extern "C" int32_t spec_distill_loss_backward(int32_t B, int32_t gamma, int32_t V, int32_t dtype,
                                              const void* draft_logits, int32_t K, const int32_t* teacher_ids,
                                              const float* teacher_values, int32_t mode, const float* temperature,
                                              const double* saved, const float* grad_loss, void* grad_out,
                                              void* stream) {
  if (!list_ok(B, gamma, V, dtype, K)) return SPEC_ERR_INVALID_ARG;
  if (mode != SPEC_DISTILL_KL && mode != SPEC_DISTILL_TV) return SPEC_ERR_INVALID_ARG;
  if (!draft_logits || !teacher_ids || !teacher_values || !temperature || !saved || !grad_loss || !grad_out)
    return SPEC_ERR_INVALID_ARG;
  if (!aligned16(draft_logits) || !aligned16(grad_out)) return SPEC_ERR_INVALID_ARG;
  DistillArgs a{};
  a.B = B; a.G = gamma; a.V = V; a.K = K; a.mode = mode;
  const int vecs = V / (dtype == SPEC_BF16 ? 8 : 4);
  a.nseg = vecs <= kSegChunk ? 1 : (vecs + kSegChunk - 1) / kSegChunk;   // a chunk each: held in registers
  const uint64_t rows = (uint64_t)B * gamma;
  if (rows * a.nseg * kSegThreads > 0xffffffffull) return SPEC_ERR_UNSUPPORTED;
  // a workgroup reads its part of the logits before it writes it; of any other place nothing is known
  const size_t bytes = rows * (size_t)V * (dtype == SPEC_BF16 ? 2 : 4), list = rows * K * sizeof(float);
  if ((grad_out != draft_logits && overlap(grad_out, bytes, draft_logits, bytes)) ||
      overlap(grad_out, bytes, teacher_ids, list) || overlap(grad_out, bytes, teacher_values, list) ||
      overlap(grad_out, bytes, saved, rows * SPEC_DISTILL_SAVED * sizeof(double)) ||
      overlap(grad_out, bytes, grad_loss, rows * sizeof(float)) ||
      overlap(grad_out, bytes, temperature, B * sizeof(float)))
    return SPEC_ERR_INVALID_ARG;
  a.draft = draft_logits; a.ids = teacher_ids; a.values = teacher_values; a.temperature = temperature;
  a.saved = const_cast<double*>(saved); a.grad_loss = grad_loss; a.grad = grad_out;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const dim3 grid((unsigned)(rows * a.nseg));
  if (dtype == SPEC_BF16) hipLaunchKernelGGL(distill_grad_kernel<true>, grid, dim3(kSegThreads), 0, s, a);
  else hipLaunchKernelGGL(distill_grad_kernel<false>, grid, dim3(kSegThreads), 0, s, a);
  return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_ERR_HIP;
}
