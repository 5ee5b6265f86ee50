// The teacher's top logits on gfx950: per draft position the K largest target logits with their
// token ids (value descending, id ascending) and ln sum_v exp(z_v / T) over the whole row.
//
// The lists stand in for the target's rows when a drafter is trained on its distributions (DSpark
// paper, §3.3), K * 8 bytes in place of V logits.  Two kernels:
//   teacher_segment_kernel -- one workgroup per (row, segment of at most 64 KB), the segment held in
//       registers (one read).  Each of the W waves takes the ceil(K / W)-th largest of its lanes' maxima; the
//       smallest of these over the waves is a bound tau that at least K values of the segment reach,
//       so the values >= tau hold the segment's K largest.  They go to the workspace as 64-bit keys
//       (ordered value, complemented id); when more than `cap` reach tau (ties, mostly) the exact
//       K-th key is found by bisection, reading the segment again (from cache), instead.  exp2 of the values against the
//       segment's maximum is summed in fp32 per thread (64 terms) and in fp64 beyond.
//   teacher_merge_kernel -- one workgroup per row drops the keys below the largest tau, sorts the
//       rest in LDS (bitonic) and writes the first K, the log normaliser and the status.
#include "common.hpp"
#include "rowseg.hpp"
#include "spec_verify.h"

namespace spec {
namespace {

constexpr int kMergeThreads = 256;
constexpr int kHitCap = 2 * SPEC_MAX_TEACHER_K + 96;   // >= list_cap
constexpr int kMergeKeys = 8192;   // keys a merge workgroup holds at most (64 KB of LDS)

struct TeacherSeg {
  double sum;     // sum of exp((z - m) / T) over the segment
  float m;        // its largest logit
  int32_t bad;    // NaN or +inf seen
  uint32_t tau;   // key that at least K of the segment's values reach (that of -inf: no bound)
  int32_t n;      // keys listed
};

struct TeacherArgs {
  int B, G, V, K, nseg, cap;
  const void* target;
  const int32_t* lengths;
  const float* temperature;
  int32_t* ids;
  float* values;
  float* lse;
  int32_t* status;
  TeacherSeg* segs;   // [B * G, nseg]
  uint64_t* keys;     // [B * G, nseg, cap]
};

__device__ __forceinline__ uint64_t pack_key(float z, int id) {
  return ((uint64_t)order_key(z + 0.f) << 32) | (uint32_t)~id;   // -0 and 0 are equal
}

struct SegShared {
  float m[kSegWaves];
  double s[kSegWaves];
  int bad[kSegWaves];
  uint32_t t[kSegWaves];
  int cnt[2][kSegWaves];
  int n, nhit;
  uint4 hit[kHitCap];     // vectors holding a value that reaches tau, and their indices
  int32_t hit_v[kHitCap];
};

template <bool BF16>
__global__ __launch_bounds__(kSegThreads) __attribute__((amdgpu_waves_per_eu(8)))
void teacher_segment_kernel(TeacherArgs a) {
  using Seg = RowSeg<BF16>;
  constexpr int EPV = Seg::EPV;
  __shared__ SegShared sh;
  const int r = (int)(blockIdx.x / (unsigned)a.nseg), seg = (int)(blockIdx.x - (unsigned)r * a.nseg);
  const int i = r / a.G, k = r - i * a.G;
  const int L = a.lengths ? a.lengths[i] : a.G;
  const float T = a.temperature[i];
  if (k >= L || L > a.G || !(T > 0.f && T < INFINITY)) return;
  const char* row = reinterpret_cast<const char*>(a.target) + ((size_t)i * (a.G + 1) + k) * (size_t)a.V * Seg::ES;
  const Seg g(row, a.V, seg, a.nseg);
  uint4 d[kSegVecs];
  g.load(row, d);
  float x = g.load_scalar(row);
  g.mask(d);
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  if (tid == 0) sh.n = sh.nhit = 0;
  float c_hi, c_lo;
  split_scale(T, c_hi, c_lo);

  float zm = x;
#pragma unroll
  for (int j = 0; j < kSegVecs; ++j) {
    float z[EPV];
    Seg::unpack(d[j], z);
#pragma unroll
    for (int e = 0; e < EPV; ++e) zm = fmaxf(zm, z[e]);
    asm volatile("" : "+v"(zm));
  }
  forget(d);
  // the wave's ceil(K / W)-th largest lane maximum, over the W waves whose lanes all hold a vector
  // (bitwise from the top; bf16 keys end at bit 16)
  const uint32_t key = order_key(zm);
  const int full = min((g.ve - g.vb) >> 6, kSegWaves);
  const int need = full ? (a.K + full - 1) / full : SPEC_WAVE + 1;
  uint32_t t = need > SPEC_WAVE ? kNegInfKey : 0xffffffffu;
  if (wave < full && need <= SPEC_WAVE) {
    t = 0;
    for (int bit = 31; bit >= (BF16 ? 16 : 0); --bit) {
      const uint32_t trial = t | (1u << bit);
      if ((int)__popcll(__ballot(key >= trial)) >= need) t = trial;
    }
    if (BF16 && t < 0x80000000u) t |= 0xffffu;
  }
  const float wm = wave_max(zm);
  if (lane == 0) {
    sh.m[wave] = wm;
    sh.t[wave] = t;
  }
  __syncthreads();
  float m = sh.m[0];
  uint32_t tau = sh.t[0];
#pragma unroll
  for (int w = 1; w < kSegWaves; ++w) {
    m = fmaxf(m, sh.m[w]);
    tau = min(tau, sh.t[w]);
  }
  const size_t slot0 = ((size_t)r * a.nseg + seg) * a.cap;
  const float tz = key_value(tau);
  float S = 0.f;
  const float mr = m > -INFINITY ? m : 0.f;   // an empty segment sums to 0
#pragma unroll
  for (int j = 0; j < kSegVecs; ++j) {
    float z[EPV];
    Seg::unpack(d[j], z);
    float s = 0.f, vm = z[0];
#pragma unroll
    for (int e = 0; e < EPV; ++e) {
      s += exp_term(z[e], mr, c_hi, c_lo);
      vm = fmaxf(vm, z[e]);
    }
    S += s;
    asm volatile("" : "+v"(S));   // one vector's values at a time: registers
    if (vm >= tz && vm > -INFINITY) {   // copied whole; its values are looked at one by one below
      const int h = atomicAdd(&sh.nhit, 1);
      if (h < kHitCap) {
        sh.hit[h] = d[j];
        sh.hit_v[h] = g.vb + j * kSegThreads + tid;
      }
    }
  }
  S += exp_term(x, mr, c_hi, c_lo);
  const int bad = !(S < INFINITY) || !(m < INFINITY);
  const double ws = wave_sum((double)S);
  const int wb = wave_or_i(bad);
  if (lane == 0) {
    sh.s[wave] = ws;
    sh.bad[wave] = wb;
  }
  __syncthreads();
  const int nhit = sh.nhit;
  auto list = [&](float z, int id) {
    if (z >= tz && z > -INFINITY) {
      const int s = atomicAdd(&sh.n, 1);
      if (s < a.cap) a.keys[slot0 + s] = pack_key(z, id);
    }
  };
  if (nhit <= kHitCap) {
    for (int h = tid; h < nhit; h += kSegThreads) {
      float z[EPV];
      Seg::unpack(sh.hit[h], z);
#pragma unroll
      for (int e = 0; e < EPV; ++e) list(z[e], g.id_of(sh.hit_v[h], e));
    }
    if (tid < g.nx) list(x, g.id_of_scalar(tid));
  }
  __syncthreads();
  int n = sh.n;
  if (n > a.cap || nhit > kHitCap) {
    // more than `cap` values reach tau: the K-th key exactly, counting over the segment again
    const uint4* vp = reinterpret_cast<const uint4*>(row + (size_t)g.head * Seg::ES);
    int step = 0;
    auto count = [&](auto pred) -> int {
      int c = tid < g.nx && pred(order_key(x + 0.f), g.id_of_scalar(tid)) ? 1 : 0;
#pragma unroll 1
      for (int v = g.vb + tid; v < g.ve; v += kSegThreads) {
        float z[EPV];
        Seg::unpack(vp[v], z);
#pragma unroll
        for (int e = 0; e < EPV; ++e) c += pred(order_key(z[e] + 0.f), g.id_of(v, e)) ? 1 : 0;
      }
      c = wave_sum_i(c);
      if (lane == 0) sh.cnt[step & 1][wave] = c;
      __syncthreads();
      int tot = 0;
#pragma unroll
      for (int w = 0; w < kSegWaves; ++w) tot += sh.cnt[step & 1][w];
      ++step;
      return tot;
    };
    uint32_t th = 0;   // the largest key that at least K values reach (n > cap >= K of them exist)
#pragma unroll 1
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t trial = th | (1u << bit);
      if (count([&](uint32_t u, int) { return u >= trial; }) >= a.K) th = trial;
    }
    const int above = count([&](uint32_t u, int) { return u > th; });
    int idb = 0;       // of the values at th, the lowest ids: ids < idb + 1
#pragma unroll 1
    for (int bit = 19; bit >= 0; --bit) {
      const int trial = idb | (1 << bit);
      if (count([&](uint32_t u, int id) { return u == th && id < trial; }) < a.K - above) idb = trial;
    }
    if (tid == 0) sh.n = 0;
    __syncthreads();
    auto take = [&](float z, int id) {
      const uint32_t u = order_key(z + 0.f);
      if (u > th || (u == th && id <= idb)) {
        const int s = atomicAdd(&sh.n, 1);
        if (s < a.cap) a.keys[slot0 + s] = pack_key(z, id);
      }
    };
#pragma unroll 1
    for (int v = g.vb + tid; v < g.ve; v += kSegThreads) {
      float z[EPV];
      Seg::unpack(vp[v], z);
#pragma unroll
      for (int e = 0; e < EPV; ++e) take(z[e], g.id_of(v, e));
    }
    if (tid < g.nx) take(x, g.id_of_scalar(tid));
    __syncthreads();
    n = min(sh.n, a.cap);
    tau = th;
  }
  if (tid == 0) {
    double s = 0.0;
    int b = 0;
#pragma unroll
    for (int w = 0; w < kSegWaves; ++w) {
      s += sh.s[w];
      b |= sh.bad[w];
    }
    a.segs[(size_t)r * a.nseg + seg] = TeacherSeg{s, mr, b, tau, n};
  }
}

__global__ __launch_bounds__(kMergeThreads) void teacher_merge_kernel(TeacherArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint64_t keys[];
  __shared__ int sbad, sn;
  const int r = (int)blockIdx.x, i = r / a.G, k = r - i * a.G, tid = threadIdx.x;
  const int L = a.lengths ? a.lengths[i] : a.G;
  const float T = a.temperature[i];
  const size_t o = (size_t)r * a.K;
  int st = 0;
  if (L < 0 || L > a.G) {
    st = SPEC_REQ_BAD_LENGTH;
  } else {
    if (!(T > 0.f && T < INFINITY)) st |= SPEC_REQ_BAD_TEMPERATURE;
    if (st == 0) {
      // every row of the request: a bad or an empty one marks the request
      if (tid == 0) sbad = sn = 0;
      __syncthreads();
      if (tid < L) {
        const TeacherSeg* p = a.segs + ((size_t)i * a.G + tid) * a.nseg;
        int bad = 0, some = 0;
        for (int s = 0; s < a.nseg; ++s) {
          bad |= p[s].bad;
          some |= p[s].sum > 0.0;
        }
        if (bad || !some) sbad = 1;
      }
      __syncthreads();
      if (sbad) st |= SPEC_REQ_NONFINITE;
    }
  }
  if (a.status && k == 0 && tid == 0) a.status[i] = st;
  if (st != 0 || k >= L) {
    const float fill = st != 0 ? NAN : -INFINITY;
    for (int e = tid; e < a.K; e += kMergeThreads) {
      a.ids[o + e] = -1;
      a.values[o + e] = fill;
    }
    if (a.lse && tid == 0) a.lse[r] = fill;
    return;
  }
  const TeacherSeg* p = a.segs + (size_t)r * a.nseg;
  uint32_t tau = kNegInfKey;
  for (int s = 0; s < a.nseg; ++s) tau = max(tau, p[s].tau);
  for (int s = 0; s < a.nseg; ++s) {
    const uint64_t* src = a.keys + ((size_t)r * a.nseg + s) * a.cap;
    for (int e = tid; e < p[s].n; e += kMergeThreads) {
      const uint64_t key = src[e];
      if ((uint32_t)(key >> 32) >= tau) keys[atomicAdd(&sn, 1)] = key;
    }
  }
  __syncthreads();
  const int n = sn;
  int N = 2;
  while (N < n) N <<= 1;
  for (int e = n + tid; e < N; e += kMergeThreads) keys[e] = 0;
  __syncthreads();
  for (int size = 2; size <= N; size <<= 1) {
    for (int stride = size >> 1; stride > 0; stride >>= 1) {
      for (int e = tid; e < N / 2; e += kMergeThreads) {
        const int lo = 2 * e - (e & (stride - 1)), hi = lo + stride;
        const uint64_t x = keys[lo], y = keys[hi];
        const bool desc = (lo & size) == 0;
        if ((x < y) == desc) {
          keys[lo] = y;
          keys[hi] = x;
        }
      }
      __syncthreads();
    }
  }
  for (int e = tid; e < a.K; e += kMergeThreads) {
    const bool on = e < n;
    const uint64_t key = on ? keys[e] : 0;
    a.ids[o + e] = on ? (int)~(uint32_t)key : -1;
    a.values[o + e] = on ? key_value((uint32_t)(key >> 32)) : -INFINITY;
  }
  if (a.lse && tid == 0) {
    float m = -INFINITY;
    for (int s = 0; s < a.nseg; ++s)
      if (p[s].sum > 0.0) m = fmaxf(m, p[s].m);
    double S = 0.0;
    for (int s = 0; s < a.nseg; ++s)
      if (p[s].sum > 0.0) S += p[s].sum * exp(((double)p[s].m - (double)m) / (double)T);
    a.lse[r] = (float)((double)m / (double)T + log(S));
  }
}

// Keys a segment may list: about K reach tau, rarely 2 K + 96; rows of one segment may have no full
// wave to take tau from (at most 64 vectors and 14 scalars, all listed then).
int list_cap(int K, int nseg) {
  const int c = 2 * K + 96 + (nseg == 1 ? 512 : 0), most = kMergeKeys / nseg;
  return c < most ? c : most;   // nseg <= 16: at least 512 >= 2 K
}

size_t workspace_of(size_t rows, int V, int K, int dtype) {
  const int nseg = row_segments(V, dtype);
  return round256(rows * nseg * sizeof(TeacherSeg)) +
         round256(rows * nseg * (size_t)list_cap(K, nseg) * sizeof(uint64_t));
}

int pow2_at_least(int n) {
  int p = 2;
  while (p < n) p <<= 1;
  return p;
}

}  // namespace
}  // namespace spec

using namespace spec;

extern "C" size_t spec_teacher_workspace_size(int32_t B, int32_t gamma, int32_t V, int32_t K) {
  if (!shape_ok(B, gamma, V, SPEC_BF16) || K < 1 || K > SPEC_MAX_TEACHER_K) return 0;
  const size_t rows = (size_t)B * gamma, b = workspace_of(rows, V, K, SPEC_BF16);
  const size_t f = V <= SPEC_MAX_V / 2 ? workspace_of(rows, V, K, SPEC_F32) : 0;
  return b > f ? b : f;
}

extern "C" int32_t spec_teacher_topk(int32_t B, int32_t gamma, int32_t V, int32_t dtype, const void* target_logits,
                                     int32_t K, const int32_t* lengths, const float* temperature, int32_t* ids_out,
                                     float* values_out, float* lse_out, int32_t* status, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  if (!shape_ok(B, gamma, V, dtype) || K < 1 || K > SPEC_MAX_TEACHER_K) return SPEC_ERR_INVALID_ARG;
  if (!target_logits || !temperature || !ids_out || !values_out) return SPEC_ERR_INVALID_ARG;
  if (!aligned16(target_logits)) return SPEC_ERR_INVALID_ARG;
  if (!workspace || !aligned256(workspace) || workspace_bytes < spec_teacher_workspace_size(B, gamma, V, K))
    return SPEC_ERR_WORKSPACE;
  TeacherArgs a{};
  a.B = B; a.G = gamma; a.V = V; a.K = K;
  a.nseg = row_segments(V, dtype);
  a.cap = list_cap(K, a.nseg);
  const uint64_t rows = (uint64_t)B * gamma;
  if (rows * a.nseg * kSegThreads > 0xffffffffull) return SPEC_ERR_UNSUPPORTED;
  a.target = target_logits; a.lengths = lengths; a.temperature = temperature;
  a.ids = ids_out; a.values = values_out; a.lse = lse_out; a.status = status;
  a.segs = reinterpret_cast<TeacherSeg*>(workspace);
  a.keys = reinterpret_cast<uint64_t*>(reinterpret_cast<char*>(workspace) +
                                       round256(rows * a.nseg * sizeof(TeacherSeg)));
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const dim3 grid((unsigned)(rows * a.nseg));
  if (dtype == SPEC_BF16)
    hipLaunchKernelGGL(teacher_segment_kernel<true>, grid, dim3(kSegThreads), 0, s, a);
  else
    hipLaunchKernelGGL(teacher_segment_kernel<false>, grid, dim3(kSegThreads), 0, s, a);
  const unsigned lds = (unsigned)(pow2_at_least(a.nseg * a.cap) * sizeof(uint64_t));
  hipLaunchKernelGGL(teacher_merge_kernel, dim3((unsigned)rows), dim3(kMergeThreads), lds, s, a);
  return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_ERR_HIP;
}
