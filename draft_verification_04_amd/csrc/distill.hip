// Distillation of the draft distribution from a teacher's top logits on gfx950, with its gradient.
//
// For a draft row z, q = softmax(z / T) over the whole row, a teacher list S of tokens with
// probabilities p_e (renormalised over the list, or scaled by the teacher's own normaliser, the rest
// r_t kept as one bucket against the draft's mass r_s outside the list):
//   KL: sum_e p_e ln(p_e / q_e) + r_t ln(r_t / r_s)
//   TV: sum_e max(p_e - q_e, 0) + max(r_t - r_s, 0)   (DSpark paper, §3.3 and Eq. 8)
// Their derivatives are multiples of q outside the list and q b - c_e in it:
//   KL: a = 1 - r_t / r_s, b = 1, c_e = p_e
//   TV: b = sum of q_e over p_e > q_e, + r_s if r_t > r_s;  a = b - [r_t > r_s];  c_e = [p_e > q_e] q_e
//   dz_v = grad_loss / T * (q_v a, or q_e b - c_e)
//
// r_s is summed over the tokens outside the list, never taken as 1 - sum of q_e: where the list holds
// nearly all of q the difference has no correct digit, and a and ln r_s hang on it.
//
// The work is one read of the rows (forward) and one read and one write (backward):
//   distill_stream_kernel -- one workgroup per (row, segment of at most 64 KB, in registers): marks the
//       listed tokens of its segment in an LDS bitmap (a byte per 16-byte vector of bf16, so a vector
//       without a listed token costs one LDS byte), takes them out and sums exp of the rest.
//   distill_finish_kernel -- one workgroup per request, a wave per row: list terms in fp64, loss,
//       the coefficients the backward reads, status.
//   distill_grad_kernel -- one workgroup per (row, segment): q a of every token as (q / r_s) (a r_s),
//       then, behind a barrier, the listed tokens' own values over it.
#include "common.hpp"
#include "rowseg.hpp"
#include "spec_verify.h"

namespace spec {
namespace {

constexpr double kLn2Seg = 0.69314718055994530942;
constexpr int kFlagBad = 1;    // NaN or +inf outside the list
constexpr int kFlagTwice = 2;  // a token id named twice
constexpr int kFlagToken = 4;  // an id outside [-1, V)
constexpr int kListWords = kSegThreads * kSegVecs * 8 / 32;   // bitmap of a bf16 segment

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
  const float* grad_loss;  // backward
  void* grad;
};

// A used entry names a token and has a logit above -inf (a NaN logit is used, and bad).
__device__ __forceinline__ bool used_entry(int id, float v) { return id != -1 && !(v == -INFINITY); }

template <bool BF16>
__global__ __launch_bounds__(kSegThreads) __attribute__((amdgpu_waves_per_eu(8)))
void distill_stream_kernel(DistillArgs a) {
  using Seg = RowSeg<BF16>;
  constexpr int EPV = Seg::EPV;
  __shared__ uint32_t bits[kListWords];
  __shared__ uint32_t xbits;
  __shared__ SegSumShared ss;
  __shared__ int sflags;
  const int r = (int)(blockIdx.x / (unsigned)a.nseg), seg = (int)(blockIdx.x - (unsigned)r * a.nseg);
  const int i = r / a.G, k = r - i * a.G;
  const int L = a.lengths ? a.lengths[i] : a.G;
  const float T = a.temperature[i];
  if (k >= L || L > a.G || !(T > 0.f && T < INFINITY)) return;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int e0 = min(tid, a.K - 1);
  const int id = a.ids[(size_t)r * a.K + e0];
  const float val = a.values[(size_t)r * a.K + e0];
  const char* row = reinterpret_cast<const char*>(a.draft) + (size_t)r * (size_t)a.V * Seg::ES;
  const Seg g(row, a.V, seg, a.nseg);
  uint4 d[kSegVecs];
  float x = g.load_scalar(row);
  g.load(row, d);
  for (int w = tid; w < kListWords; w += kSegThreads) bits[w] = 0;
  if (tid == 0) xbits = sflags = 0;
  lds_barrier();
  if (tid < a.K && used_entry(id, val)) {
    if (id < 0 || id >= a.V) {
      if (seg == 0) atomicOr(&sflags, kFlagToken);
    } else {
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
  }
  lds_barrier();
  float c_hi, c_lo;
  split_scale(T, c_hi, c_lo);
  if (tid < g.nx && ((xbits >> tid) & 1u)) x = -INFINITY;
  RunningSum sum{kNoReference, 0.f, 0};
  const uint8_t* bytes = reinterpret_cast<const uint8_t*>(bits);
  // vector j without its listed tokens
  auto unlisted = [&](uint4 v, int j) -> uint4 {
    const int lv = j * kSegThreads + tid;
    uint32_t w;
    if constexpr (BF16) w = bytes[lv];
    else w = (bytes[lv >> 1] >> ((lv & 1) * 4)) & 15u;
    if (w) {
      if constexpr (BF16) {
        uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int h = 0; h < 4; ++h) {
          if (w & (1u << (2 * h))) q[h] = (q[h] & 0xffff0000u) | 0xff80u;
          if (w & (2u << (2 * h))) q[h] = (q[h] & 0xffffu) | 0xff800000u;
        }
        v = make_uint4(q[0], q[1], q[2], q[3]);
      } else {
        if (w & 1u) v.x = 0xff800000u;
        if (w & 2u) v.y = 0xff800000u;
        if (w & 4u) v.z = 0xff800000u;
        if (w & 8u) v.w = 0xff800000u;
      }
    }
    return v;
  };
#pragma unroll
  for (int j = 0; j < kSegVecs; ++j) {
    if (g.vb + j * kSegThreads < g.ve) {
      uint4 v = unlisted(d[j], j);
      if (g.vb + j * kSegThreads + tid >= g.ve) v = make_uint4(Seg::kNegInf, Seg::kNegInf, Seg::kNegInf, Seg::kNegInf);
      float z[EPV];
      Seg::unpack(v, z);
      add_terms<EPV>(sum, z, c_hi, c_lo);
    }
    asm volatile("" : "+v"(sum.S));   // one vector's values at a time: registers
  }
  if (g.nx > 0) {
    const float z1[1] = {x};
    add_terms<1>(sum, z1, c_hi, c_lo);
  }
  int bad;
  const SegSum t = segment_sum<BF16>(ss, sum, [&](int j) { return unlisted(g.reload(row, j), j); }, x, c_hi, c_lo, bad);
  if (tid == 0) a.segs[(size_t)r * a.nseg + seg] = DistillSeg{t.sum, t.ref, sflags | (bad ? kFlagBad : 0), 0};
}

__device__ __forceinline__ double wave_max_d(double x) {
  return wave_reduce(x, [](double p, double q) { return fmax(p, q); });
}

// Waves of a workgroup at most; entries of a list per lane (one for K <= 64, else four).
constexpr int finish_waves(int entries) { return entries == 1 ? 16 : 8; }

template <bool BF16, int kLaneEntries>
__global__ __launch_bounds__(finish_waves(kLaneEntries) * SPEC_WAVE) void distill_finish_kernel(DistillArgs a) {
  __shared__ int sst;
  const int i = (int)blockIdx.x, tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int nw = (int)blockDim.x >> 6;
  const int G = a.G, K = a.K, V = a.V;
  const int L = a.lengths ? a.lengths[i] : G;
  const float T = a.temperature[i];
  int st = 0;
  if (L < 0 || L > G) st = SPEC_REQ_BAD_LENGTH;
  else if (!(T > 0.f && T < INFINITY)) st = SPEC_REQ_BAD_TEMPERATURE;
  if (tid == 0) sst = st;
  __syncthreads();
  const double Td = (double)T;
  for (int k = wave; k < G; k += nw) {
    const size_t r = (size_t)i * G + k;
    double* sv = a.saved + r * SPEC_DISTILL_SAVED;
    bool live = st == 0 && k < L;
    double loss = 0.0;
    if (live) {
      // every load of the row at once: a lane's entries, and a segment per lane (at most 16)
      const DistillSeg* p = a.segs + r * a.nseg;
      int id[kLaneEntries];
      float val[kLaneEntries];
#pragma unroll
      for (int u = 0; u < kLaneEntries; ++u) {
        const int e = min(lane + u * SPEC_WAVE, K - 1);
        id[u] = a.ids[r * K + e];
        val[u] = a.values[r * K + e];
      }
      const DistillSeg mine = p[min(lane, a.nseg - 1)];
      const float tl = a.teacher_lse ? a.teacher_lse[r] : 0.f;
      int rst = 0, any = 0, nused = 0;
      float zv[kLaneEntries];
#pragma unroll
      for (int u = 0; u < kLaneEntries; ++u) {
        const bool used = lane + u * SPEC_WAVE < K && used_entry(id[u], val[u]);
        any |= used;
        if (used && (id[u] < 0 || id[u] >= V)) rst |= SPEC_REQ_BAD_TOKEN;
        if (!used || id[u] < 0 || id[u] >= V) id[u] = -1;
        zv[u] = load_elem<BF16>(reinterpret_cast<const char*>(a.draft) + r * (size_t)V * (BF16 ? 2 : 4),
                                max(id[u], 0));
      }
      live = __ballot(any) != 0;
      if (live) {
        const double c = kLog2eSeg / Td;   // exponents in powers of two
        double tv[kLaneEntries], zq[kLaneEntries], tmax = -INFINITY, zmax = -INFINITY;
#pragma unroll
        for (int u = 0; u < kLaneEntries; ++u) {
          const bool on = id[u] >= 0;
          if (on && (!(val[u] < INFINITY) || !(zv[u] < INFINITY))) rst |= SPEC_REQ_NONFINITE;
          nused += on;
          tv[u] = on ? (double)val[u] * c : -INFINITY;
          zq[u] = on ? (double)zv[u] * c : -INFINITY;
          tmax = fmax(tmax, tv[u]);
          zmax = fmax(zmax, zq[u]);
        }
        const bool seg_on = lane < a.nseg && mine.sum > 0.0;
        if (lane < a.nseg) {
          if (mine.flags & kFlagBad) rst |= SPEC_REQ_NONFINITE;
          if (mine.flags & kFlagToken) rst |= SPEC_REQ_BAD_TOKEN;
          if (mine.flags & kFlagTwice) rst |= SPEC_REQ_BAD_LIST;
        }
        // outside the list: out * 2^mo, lo its log2
        const double mo = wave_max_d(seg_on ? mine.ref : -INFINITY);
        const bool outside = mo > -INFINITY;
        tmax = wave_max_d(tmax);
        zmax = fmax(wave_max_d(zmax), mo);
        nused = wave_sum_i(nused);
        const bool tail = a.teacher_lse != nullptr;
        if (tail && !(fabsf(tl) < INFINITY)) rst |= SPEC_REQ_NONFINITE;
        if (!(zmax > -INFINITY)) rst |= SPEC_REQ_NONFINITE;
        rst = wave_or_i(rst);
        if (rst == 0) {
          const double out = wave_sum(seg_on ? mine.sum * exp2(mine.ref - mo) : 0.0);
          double el[kLaneEntries], te[kLaneEntries], lsum = 0.0, tsum = 0.0;
#pragma unroll
          for (int u = 0; u < kLaneEntries; ++u) {
            el[u] = te[u] = 0.0;
            if (u * SPEC_WAVE < K) {
              el[u] = exp2(zq[u] - zmax);
              te[u] = exp2(tv[u] - tmax);
            }
            lsum += el[u];
            tsum += te[u];
          }
          lsum = wave_sum(lsum);
          tsum = wave_sum(tsum);
          // in logs: the tail may lie hundreds of nats below the list
          const double lo = outside ? mo - zmax + log2(out) : -INFINITY;
          const double tot = exp2(lo) + lsum, lt = log2(tot);
          const double t = tail ? (double)tl * kLog2eSeg : tmax + log2(tsum);   // log2 of p's normaliser
          const double ps = exp2(tmax - t);
          const double lrs = lo - lt, rs = exp2(lrs);
          const double rt = (tail && nused < V) ? fmax(0.0, 1.0 - tsum * ps) : 0.0;
          double ars, bv;   // a r_s: q a = (q / r_s) (a r_s) outside the list, finite however small r_s
          double sum = 0.0, qs = 0.0;
#pragma unroll
          for (int u = 0; u < kLaneEntries; ++u) {
            if (id[u] < 0) continue;
            const double pe = te[u] * ps, qe = el[u] / tot;
            if (a.mode == SPEC_DISTILL_KL) {
              if (pe > 0.0) sum += pe * ((tv[u] - t) - (zq[u] - zmax - lt));
            } else if (pe > qe) {
              sum += pe - qe;
              qs += qe;
            }
          }
          loss = wave_sum(sum);
          if (a.mode == SPEC_DISTILL_KL) {
            bv = 1.0;
            ars = rs - rt;
            if (rt > 0.0) loss += rt * (log2(rt) - lrs);   // +inf when the draft leaves no mass there
            loss *= kLn2Seg;
          } else {
            const bool up = rt > rs;
            if (up) loss += rt - rs;
            bv = wave_sum(qs) + (up ? rs : 0.0);
            ars = (bv - (up ? 1.0 : 0.0)) * rs;
          }
          if (lane == 0) {
            // q / r_s = exp2((z - m) c - sv[1]): the logit nearest the largest exponent as reference
            const float m = outside ? (float)(mo / c) : 0.f;
            sv[0] = (double)m;
            sv[1] = outside ? mo - (double)m * c + log2(out) : 0.0;
            sv[2] = outside ? ars : 0.0;
            sv[3] = bv;
            sv[4] = t;
            sv[5] = zmax + lt;
          }
        } else if (lane == 0) {
          atomicOr(&sst, rst);
        }
      }
    }
    if (lane == 0) {
      a.loss[r] = (float)loss;
      if (!live) sv[0] = NAN;
    }
  }
  __syncthreads();
  st = sst;
  if (tid == 0 && a.status) a.status[i] = st;
  if (st)
    for (int k = tid; k < G; k += (int)blockDim.x) {
      a.loss[(size_t)i * G + k] = NAN;
      a.saved[((size_t)i * G + k) * SPEC_DISTILL_SAVED] = NAN;
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
  const float f = (float)(s * sv[2]);
  // every load of the segment is done in every wave before the first store (grad may be draft)
  memory_barrier();
  auto grad_of = [&](float z) {
    const float dz = z - m;   // q / r_s of a token outside the list
    return f * __builtin_amdgcn_exp2f(fmaf(dz, c_lo, fmaf(dz, c_hi, -l2)));
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
    const double Td = (double)T;
    const double c2 = kLog2eSeg / Td;
    const double q = exp2((double)ze * c2 - sv[5]), p = exp2((double)val * c2 - sv[4]);
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
  return round256((size_t)B * gamma * row_segments(V, SPEC_F32) * sizeof(DistillSeg));
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
  a.nseg = row_segments(V, dtype);
  const uint64_t rows = (uint64_t)B * gamma;
  if (rows * a.nseg * kSegThreads > 0xffffffffull) return SPEC_ERR_UNSUPPORTED;
  const int entries = K <= SPEC_WAVE ? 1 : SPEC_MAX_TEACHER_K / SPEC_WAVE;
  const int waves = gamma < finish_waves(entries) ? gamma : finish_waves(entries);
  if ((uint64_t)B * waves * SPEC_WAVE > 0xffffffffull) return SPEC_ERR_UNSUPPORTED;
  a.draft = draft_logits; a.ids = teacher_ids; a.values = teacher_values; a.teacher_lse = teacher_lse;
  a.lengths = lengths; a.temperature = temperature; a.loss = loss_out; a.saved = saved_out; a.status = status;
  a.segs = reinterpret_cast<DistillSeg*>(workspace);
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const dim3 grid((unsigned)(rows * a.nseg)), fgrid((unsigned)B), fblock((unsigned)(waves * SPEC_WAVE));
  if (dtype == SPEC_BF16) {
    hipLaunchKernelGGL(distill_stream_kernel<true>, grid, dim3(kSegThreads), 0, s, a);
    if (entries == 1) hipLaunchKernelGGL((distill_finish_kernel<true, 1>), fgrid, fblock, 0, s, a);
    else hipLaunchKernelGGL((distill_finish_kernel<true, 4>), fgrid, fblock, 0, s, a);
  } else {
    hipLaunchKernelGGL(distill_stream_kernel<false>, grid, dim3(kSegThreads), 0, s, a);
    if (entries == 1) hipLaunchKernelGGL((distill_finish_kernel<false, 1>), fgrid, fblock, 0, s, a);
    else hipLaunchKernelGGL((distill_finish_kernel<false, 4>), fgrid, fblock, 0, s, a);
  }
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
  a.nseg = row_segments(V, dtype);
  const uint64_t rows = (uint64_t)B * gamma;
  if (rows * a.nseg * kSegThreads > 0xffffffffull) return SPEC_ERR_UNSUPPORTED;
  a.draft = draft_logits; a.ids = teacher_ids; a.values = teacher_values; a.temperature = temperature;
  a.saved = const_cast<double*>(saved); a.grad_loss = grad_loss; a.grad = grad_out;
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const dim3 grid((unsigned)(rows * a.nseg));
  if (dtype == SPEC_BF16) hipLaunchKernelGGL(distill_grad_kernel<true>, grid, dim3(kSegThreads), 0, s, a);
  else hipLaunchKernelGGL(distill_grad_kernel<false>, grid, dim3(kSegThreads), 0, s, a);
  return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_ERR_HIP;
}
