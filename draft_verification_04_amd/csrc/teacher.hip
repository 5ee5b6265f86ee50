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
//       K-th key is found by bisection, reading the segment again (from cache), instead.  The terms
//       exp(z / T) are summed in fp32 per thread (64 terms) and in fp64 beyond.
//   teacher_merge_kernel -- one wave per row drops the keys below the largest tau, keeps the K largest
//       of the rest in order, and writes them, the log normaliser and the status.
#include "common.hpp"
#include "rowseg.hpp"
#include "spec_verify.h"

namespace spec {
namespace {

constexpr int kHitCap = 3 * SPEC_MAX_TEACHER_K + 96;
constexpr int kMergeWaves = 4;      // rows per workgroup of the merge
constexpr int kMergeRegs = 32;      // keys of the lists a lane of it holds at most

struct TeacherSeg {
  double sum, ref;  // sum of exp(z / T) over the segment: sum * 2^ref
  int32_t bad;      // NaN or +inf seen
  uint32_t tau;     // key that at least K of the segment's values reach (that of -inf: no bound)
  int32_t n, pad;   // keys listed
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
  SegSumShared sum;
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
  const float x = g.load_scalar(row);
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  if (tid == 0) sh.n = sh.nhit = 0;
  float c_hi, c_lo;
  split_scale(T, c_hi, c_lo);

  RunningSum sum{kNoReference, 0.f, 0};
  float vm[kSegVecs], zm = x;   // the vectors' largest values
#pragma unroll
  for (int j = 0; j < kSegVecs; ++j) {
    vm[j] = -INFINITY;
    if (g.vb + j * kSegThreads < g.ve) {
      uint4 v = d[j];
      if (g.vb + j * kSegThreads + tid >= g.ve) v = make_uint4(Seg::kNegInf, Seg::kNegInf, Seg::kNegInf, Seg::kNegInf);
      float z[EPV];
      Seg::unpack(v, z);
      add_terms<EPV>(sum, z, c_hi, c_lo);
      vm[j] = z[0];
#pragma unroll
      for (int e = 1; e < EPV; ++e) vm[j] = fmaxf(vm[j], z[e]);
      zm = fmaxf(zm, vm[j]);
    }
    asm volatile("" : "+v"(sum.S), "+v"(vm[j]));   // one vector's values at a time: registers
  }
  if (g.nx > 0) {
    const float z1[1] = {x};
    add_terms<1>(sum, z1, c_hi, c_lo);
  }
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
  if (lane == 0) sh.t[wave] = t;
  __syncthreads();
  uint32_t tau = sh.t[0];
#pragma unroll
  for (int w = 1; w < kSegWaves; ++w) tau = min(tau, sh.t[w]);
  const size_t slot0 = ((size_t)r * a.nseg + seg) * a.cap;
  const float tz = key_value(tau);
#pragma unroll
  for (int j = 0; j < kSegVecs; ++j) {
    if (vm[j] >= tz && vm[j] > -INFINITY) {   // copied whole; its values are looked at one by one below
      const int h = atomicAdd(&sh.nhit, 1);
      if (h < kHitCap) {
        sh.hit[h] = d[j];
        sh.hit_v[h] = g.vb + j * kSegThreads + tid;
      }
    }
  }
  int bad;
  const SegSum total = segment_sum<BF16>(sh.sum, sum, [&](int j) { return g.reload(row, j); }, x, c_hi, c_lo, bad);
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
  if (tid == 0) a.segs[(size_t)r * a.nseg + seg] = TeacherSeg{total.sum, total.ref, bad, tau, n, 0};
}

__device__ __forceinline__ double wave_max_d(double x) {
  return wave_reduce(x, [](double p, double q) { return fmax(p, q); });
}

// One wave per row.  The keys kept so far and as many segments' lists as fit are held in registers; the K-th largest value is found bit by bit, of the values equal
// to it the lowest ids, and the survivors go to LDS.  In the end every key's place is the number of
// larger ones.
__global__ __launch_bounds__(kMergeWaves * SPEC_WAVE) void teacher_merge_kernel(TeacherArgs a, int key_bits) {
  __shared__ uint64_t kept[kMergeWaves][SPEC_MAX_TEACHER_K];
  const int wave = (int)threadIdx.x >> 6, lane = (int)threadIdx.x & 63;
  const long long row = (long long)blockIdx.x * kMergeWaves + wave;
  if (row >= (long long)a.B * a.G) return;
  const int r = (int)row, i = r / a.G, k = r - i * a.G, K = a.K;
  const int L = a.lengths ? a.lengths[i] : a.G;
  const float T = a.temperature[i];
  const size_t o = (size_t)r * K;
  const TeacherSeg* p = a.segs + (size_t)r * a.nseg;
  int st = 0;
  if (L < 0 || L > a.G) st = SPEC_REQ_BAD_LENGTH;
  else if (!(T > 0.f && T < INFINITY)) st = SPEC_REQ_BAD_TEMPERATURE;
  if (st == 0 && L > 0) {
    // every row of the request: a bad or an empty one marks the request
    const TeacherSeg* q = a.segs + ((size_t)i * a.G + min(lane, L - 1)) * a.nseg;
    int bad = 0, some = 0;
    for (int s = 0; s < a.nseg; ++s) {
      bad |= q[s].bad;
      some |= q[s].sum > 0.0;
    }
    if (__ballot(bad || !some)) st = SPEC_REQ_NONFINITE;
  }
  if (a.status && k == 0 && lane == 0) a.status[i] = st;
  if (st != 0 || k >= L) {
    const float fill = st != 0 ? NAN : -INFINITY;
    for (int e = lane; e < K; e += SPEC_WAVE) {
      a.ids[o + e] = -1;
      a.values[o + e] = fill;
    }
    if (a.lse && lane == 0) a.lse[r] = fill;
    return;
  }
  const TeacherSeg mine = p[min(lane, a.nseg - 1)];   // nseg <= 16
  const bool on = lane < a.nseg;
  const uint32_t tau = (uint32_t)wave_max_i(on ? (int)(mine.tau ^ 0x80000000u) : INT32_MIN) ^ 0x80000000u;
  uint64_t* list = kept[wave];
  int cur = 0, s0 = 0;
  constexpr int KR = SPEC_MAX_TEACHER_K / SPEC_WAVE;   // registers of the keys kept so far
  while (s0 < a.nseg) {
    // a round: registers 0 .. KR - 1 hold the kept keys, each further one 64 keys of one segment's list
    uint32_t hi[KR + kMergeRegs], lo[KR + kMergeRegs];
#pragma unroll
    for (int u = 0; u < KR; ++u) {
      const uint64_t key = lane + u * SPEC_WAVE < cur ? list[lane + u * SPEC_WAVE] : 0;
      hi[u] = (uint32_t)(key >> 32);
      lo[u] = (uint32_t)key;
    }
    int used = 0, s1 = s0;
    while (s1 < a.nseg) {
      const int n = max(1, (read_lane(mine.n, s1) + SPEC_WAVE - 1) / SPEC_WAVE);   // an empty one takes a register too
      if (used + n > kMergeRegs) break;
      used += n;
      ++s1;
    }
    int s = s0, off = 0;
#pragma unroll
    for (int g = 0; g < kMergeRegs; g += 8) {
      if (g < used) {   // eight loads at once, clamped in bounds
        uint64_t key[8];
        bool in[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const int sc = min(s, s1 - 1), n = read_lane(mine.n, sc), e = off + lane;
          in[u] = s < s1 && e < n;
          key[u] = a.keys[((size_t)r * a.nseg + sc) * a.cap + min(e, a.cap - 1)];
          off += SPEC_WAVE;
          if (off >= n) {
            off = 0;
            ++s;
          }
        }
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          const bool take = in[u] && (uint32_t)(key[u] >> 32) >= tau;
          hi[KR + g + u] = take ? (uint32_t)(key[u] >> 32) : 0;
          lo[KR + g + u] = (uint32_t)key[u];
        }
      } else {
#pragma unroll
        for (int u = 0; u < 8; ++u) hi[KR + g + u] = lo[KR + g + u] = 0;
      }
    }
    auto count = [&](auto pred) -> int {
      int c = 0;
      if (cur > 0) {
#pragma unroll
        for (int u = 0; u < KR; ++u) c += (int)__popcll(__ballot(pred(hi[u], lo[u])));
      }
#pragma unroll
      for (int g = 0; g < kMergeRegs; g += 8)
        if (g < used) {
#pragma unroll
          for (int u = KR + g; u < KR + g + 8; ++u) c += (int)__popcll(__ballot(pred(hi[u], lo[u])));
        }
      return c;
    };
    uint32_t th = 0;   // the largest value key that at least K keys reach (0: fewer than K keys)
#pragma unroll 1
    for (int bit = 31; bit >= 32 - key_bits; --bit) {
      const uint32_t trial = th | (1u << bit);
      if (count([&](uint32_t h, uint32_t) { return h >= trial; }) >= K) th = trial;
    }
    uint32_t tl = 0;   // of the keys at th, the largest low words (lowest ids) that fill up K
    // bf16 keys of negative values end in 16 ones: th stands for them with zeros there
    const uint32_t top = th | (key_bits < 32 ? 0xffffu : 0u);
    if (th > 0) {
      const int above = count([&](uint32_t h, uint32_t) { return h > top; });
      if (count([&](uint32_t h, uint32_t) { return h >= th; }) > K) {
        tl = 0xfff00000u;
#pragma unroll 1
        for (int bit = 19; bit >= 0; --bit) {
          const uint32_t trial = tl | (1u << bit);
          if (count([&](uint32_t h, uint32_t l) { return h >= th && h <= top && l >= trial; }) >= K - above) tl = trial;
        }
      }
    }
    int kept_n = 0;
#pragma unroll
    for (int u = 0; u < KR + kMergeRegs; ++u) {
      if (u < KR ? cur > 0 : u - KR < used) {
        const bool take = hi[u] > 0 && (hi[u] > top || (hi[u] >= th && lo[u] >= tl));
        const unsigned long long m = __ballot(take);
        const int e = kept_n + (int)__popcll(m & ((1ull << lane) - 1));
        if (take && e < SPEC_MAX_TEACHER_K) list[e] = ((uint64_t)hi[u] << 32) | lo[u];
        kept_n += (int)__popcll(m);
      }
    }
    cur = min(kept_n, K);
    s0 = s1;
  }
  uint64_t key[SPEC_MAX_TEACHER_K / SPEC_WAVE];
  int place[SPEC_MAX_TEACHER_K / SPEC_WAVE];
#pragma unroll
  for (int u = 0; u < SPEC_MAX_TEACHER_K / SPEC_WAVE; ++u) {
    key[u] = lane + u * SPEC_WAVE < cur ? list[lane + u * SPEC_WAVE] : 0;
    place[u] = 0;
  }
  if (cur <= SPEC_WAVE) {
#pragma unroll 8
    for (int e = 0; e < cur; ++e) place[0] += list[e] > key[0] ? 1 : 0;
  } else {
#pragma unroll 4
    for (int e = 0; e < cur; ++e) {
      const uint64_t x = list[e];
#pragma unroll
      for (int u = 0; u < SPEC_MAX_TEACHER_K / SPEC_WAVE; ++u) place[u] += x > key[u] ? 1 : 0;
    }
  }
#pragma unroll
  for (int u = 0; u < SPEC_MAX_TEACHER_K / SPEC_WAVE; ++u) {
    const int e = lane + u * SPEC_WAVE;
    if (e < cur) {
      a.ids[o + place[u]] = (int)~(uint32_t)key[u];
      a.values[o + place[u]] = key_value((uint32_t)(key[u] >> 32));
    } else if (e < K) {
      a.ids[o + e] = -1;
      a.values[o + e] = -INFINITY;
    }
  }
  if (a.lse) {
    const bool some = on && mine.sum > 0.0;
    const double ref = wave_max_d(some ? mine.ref : -INFINITY);
    const double S = wave_sum(some ? mine.sum * exp2(mine.ref - ref) : 0.0);
    if (lane == 0) a.lse[r] = (float)(0.69314718055994530942 * (ref + log2(S)));
  }
}

// Keys a segment may list: 22 (K = 1) to 460 (K = 256) reach tau on Gaussian rows, 700 at most seen of
// 160 segments; rows of one segment may have no full wave to take tau from (at most 64 vectors and 14
// scalars, all listed then).
int list_cap(int K, int nseg) { return 3 * K + 96 + (nseg == 1 ? 512 : 0); }
static_assert(3 * SPEC_MAX_TEACHER_K + 96 + 512 <= SPEC_WAVE * kMergeRegs, "a segment's list fits a round");

size_t workspace_of(size_t rows, int V, int K, int dtype) {
  const int nseg = row_segments(V, dtype);
  return round256(rows * nseg * sizeof(TeacherSeg)) +
         round256(rows * nseg * (size_t)list_cap(K, nseg) * sizeof(uint64_t));
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
  hipLaunchKernelGGL(teacher_merge_kernel, dim3((unsigned)((rows + kMergeWaves - 1) / kMergeWaves)),
                     dim3(kMergeWaves * SPEC_WAVE), 0, s, a, dtype == SPEC_BF16 ? 16 : 32);
  return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_ERR_HIP;
}
