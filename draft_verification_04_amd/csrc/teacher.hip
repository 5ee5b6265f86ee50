// The teacher's top logits on gfx950: per draft position the K largest target logits with their
// token ids (value descending, id ascending) and ln sum_v exp(z_v / T) over the whole row.
//
// The lists stand in for the target's rows when a drafter is trained on its distributions (DSpark
// paper, §3.3), K * 8 bytes in place of V logits.  The work is one read of the rows:
//   teacher_row_kernel -- one workgroup per row (or segment of one, when there are few rows).  A bound
//       tau that at least K values reach comes from the lanes' running maxima: each of the W waves takes
//       the ceil(K / W)-th largest of its lanes', tau is the smallest of these, and it is raised after
//       the chunks 1, 2, 4 (so about 1.8 K values reach tau per doubling of what was read).  A vector
//       holding a value >= tau is copied to LDS whole; in the end the candidates >= the last tau are
//       listed (about 1.8 K), and of a whole row one wave finds the K-th largest among them bit by bit
//       (select_topk) and the survivors are put in order by counting.  Where too many values reach tau (ties,
//       rising rows) the K-th key is found by counting over the row again instead.  The terms
//       exp(z / T) are summed on the way, fp32 per thread and fp64 beyond.
//   teacher_merge_kernel -- one workgroup per row: the same selection over the lists of a row's segments;
//       and, also for whole rows, the status of the request.
//
// Bound by the read of the rows where there are many (MI355X: 256 x 16 rows of 151936 bf16, half of them live,
// K = 64: 110-122 us, 5.1-5.6 TB/s).  672 rows of 129280 with K = 256 take 55 us, 3.2 TB/s: every row is in
// flight at once, so the chip waits while all of them start (6 us) and select (12 us: listing 3, the K-th
// largest 5, the order 3).  The selection's loops kept in registers and unrolled took as long: such code runs
// once per row and is fetched cold.
#include "common.hpp"
#include "rowseg.hpp"
#include "spec_verify.h"

namespace spec {
namespace {

constexpr int kMergeKeys = 4096;   // keys of a round of the merge

struct TeacherSeg {
  double sum, ref;  // sum of exp(z / T) over the segment: sum * 2^ref
  int32_t bad;      // NaN or +inf seen
  uint32_t tau;     // key that at least K of the segment's values reach (that of -inf: no bound)
  int32_t n, pad;   // keys listed
};

struct TeacherArgs {
  int B, G, V, K, nseg, cap, hits;
  const void* target;
  const int32_t* lengths;
  const float* temperature;
  int32_t* ids;
  float* values;
  float* lse;
  int32_t* status;
  TeacherSeg* segs;   // [B * G, nseg]
  uint64_t* keys;     // [B * G, nseg, cap] (several segments)
};

// Ordered value (-0 and 0 are equal) above the complemented id: larger keys come first.
__device__ __forceinline__ uint64_t pack_key(float z, int id) {
  return ((uint64_t)order_key(z + 0.f) << 32) | (uint32_t)~id;
}

struct SelectShared {
  int cnt[2][kSegWaves];   // of the counts over a row
  int n;
  uint32_t tie[SPEC_WAVE];
  uint64_t list[SPEC_MAX_TEACHER_K];
  int place[SPEC_MAX_TEACHER_K];
};

// One wave: keeps the K largest of the n keys (distinct) in LDS, in any order, in sh.list, and their number in
// sh.n.  One wave, not eight: a few hundred keys are a few per lane, and a step costs a wave the same
// whatever it holds.  Value keys are compared without their low SH bits (16 for bf16, whose keys end
// there).  floor_key: a value key that no key lies below.
template <int SH>
__device__ __forceinline__ void select_topk(SelectShared& sh, const uint64_t* keys, int n, int K, uint32_t floor_key) {
  const int lane = (int)threadIdx.x & 63;
  const uint32_t* words = reinterpret_cast<const uint32_t*>(keys);   // low word (id), high word (value)
  constexpr int U = 8, R = U * SPEC_WAVE;   // keys in registers; the others are read from LDS again and again
  // value words (0: no key; every key's is larger) and id words of keys e, e + 64, ..
  auto fetch = [&](int e, uint32_t (&h)[U], uint32_t (&l)[U]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = min(e + u * SPEC_WAVE, n - 1);
      h[u] = e + u * SPEC_WAVE < n ? words[2 * at + 1] >> SH : 0;
      l[u] = words[2 * at];
    }
  };
  uint32_t h0[U], l0[U];
  if (n > 0) fetch(lane, h0, l0);
  auto count = [&](auto pred) -> int {
    int c = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) c += (int)__popcll(__ballot(pred(h0[u], l0[u])));
#pragma unroll 1
    for (int e = R + lane; e - lane < n; e += R) {
      uint32_t h[U], l[U];
      fetch(e, h, l);
#pragma unroll
      for (int u = 0; u < U; ++u) c += (int)__popcll(__ballot(pred(h[u], l[u])));
    }
    return c;
  };
  uint32_t th = 0, tl = 0;
  if (n > K) {
    // the largest value key that at least K keys reach; the bits above the highest one in which the keys
    // differ are known
    uint32_t top = 0;
    for (int e = lane; e < n; e += SPEC_WAVE) top = max(top, words[2 * e + 1] >> SH);
    top = (uint32_t)wave_max_i((int)(top ^ 0x80000000u)) ^ 0x80000000u;
    const uint32_t low = floor_key >> SH;
    const int high = top == low ? -1 : 31 - __clz((int)(top ^ low));
    th = high < 0 ? top : (top >> high >> 1) << high << 1;
    int reach = n;
#pragma unroll 1
    for (int bit = high; bit >= 0 && reach != K; --bit) {
      const uint32_t trial = th | (1u << bit);
      const int c = count([&](uint32_t h, uint32_t) { return h >= trial; });
      if (c >= K) {
        th = trial;
        reach = c;
      }
    }
    if (reach > K) {   // of the keys at th the largest low words (lowest ids) that fill up K
      const int above = count([&](uint32_t h, uint32_t) { return h > th; }), need = K - above;
      if (reach - above <= SPEC_WAVE) {   // a key per lane, its place by counting
        int m = 0;
#pragma unroll 1
        for (int e = lane; e - lane < n; e += SPEC_WAVE) {
          const int at = min(e, n - 1);
          const bool tie = e < n && words[2 * at + 1] >> SH == th;
          const unsigned long long b = __ballot(tie);
          if (tie) sh.tie[m + (int)__popcll(b & ((1ull << lane) - 1))] = words[2 * at];
          m += (int)__popcll(b);
        }
        const uint32_t mine = lane < m ? sh.tie[lane] : 0;
        int before = 0;
#pragma unroll 4
        for (int e = 0; e < m; ++e) before += sh.tie[e] > mine ? 1 : 0;
        const unsigned long long last = __ballot(lane < m && before == need - 1);
        tl = read_lane(mine, (int)__ffsll((long long)last) - 1);
      } else {
        tl = 0xfff00000u;
#pragma unroll 1
        for (int bit = 19; bit >= 0; --bit) {
          const uint32_t trial = tl | (1u << bit);
          const int c = count([&](uint32_t h, uint32_t l) { return h == th && l >= trial; });
          if (c >= need) tl = trial;
          if (c == need) break;
        }
      }
    }
  }
  int kept = 0;
#pragma unroll 1
  for (int e = lane; e - lane < n; e += SPEC_WAVE) {
    const uint64_t key = keys[min(e, n - 1)];
    const uint32_t h = (uint32_t)(key >> 32) >> SH;
    const bool take = e < n && (h > th || (h == th && (uint32_t)key >= tl));
    const unsigned long long m = __ballot(take);
    const int at = kept + (int)__popcll(m & ((1ull << lane) - 1));
    if (take && at < SPEC_MAX_TEACHER_K) sh.list[at] = key;
    kept += (int)__popcll(m);
  }
  if (lane == 0) sh.n = min(kept, K);
}

// Writes the sh.n selected keys of row r in order, unused entries behind them: a key's place is the number
// of larger ones, counted by the workgroup's waves (NW) in slices of the list, 64 keys at a time.
template <int NW>
__device__ __forceinline__ void write_list(SelectShared& sh, const TeacherArgs& a, int r) {
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, n = sh.n;
  const int groups = max(1, (n + SPEC_WAVE - 1) / SPEC_WAVE), slices = NW / groups;   // n <= 256: 4 groups
  static_assert(NW >= SPEC_MAX_TEACHER_K / SPEC_WAVE, "a wave per 64 keys");
  for (int e = tid; e < n; e += NW * SPEC_WAVE) sh.place[e] = 0;
  __syncthreads();
  const int grp = wave % groups, slice = wave / groups, e = grp * SPEC_WAVE + lane;
  if (slice < slices && e < n) {
    const uint64_t mine = sh.list[e];
    int before = 0;
#pragma unroll 4
    for (int f = n * slice / slices; f < n * (slice + 1) / slices; ++f) before += sh.list[f] > mine ? 1 : 0;
    atomicAdd(&sh.place[e], before);
  }
  __syncthreads();
  const size_t o = (size_t)r * a.K;
  if (tid < n) {
    const uint64_t key = sh.list[tid];
    a.ids[o + sh.place[tid]] = (int)~(uint32_t)key;
    a.values[o + sh.place[tid]] = key_value((uint32_t)(key >> 32));
  } else if (tid < a.K) {
    a.ids[o + tid] = -1;
    a.values[o + tid] = -INFINITY;
  }
}

__device__ __forceinline__ void write_empty(const TeacherArgs& a, int r, float fill) {
  const size_t o = (size_t)r * a.K;
  for (int e = threadIdx.x; e < a.K; e += (int)blockDim.x) {
    a.ids[o + e] = -1;
    a.values[o + e] = fill;
  }
  if (a.lse && threadIdx.x == 0) a.lse[r] = fill;
}

struct RowShared {
  LiveShared live;
  SegSumShared sum;
  SelectShared sel;
  uint32_t t[2][kSegWaves];
  int n, nhit;
};

template <bool BF16>
__global__ __launch_bounds__(kSegThreads) __attribute__((amdgpu_waves_per_eu(8)))
void teacher_row_kernel(TeacherArgs a) {
  using Seg = RowSeg<BF16>;
  constexpr int EPV = Seg::EPV;
  extern __shared__ __attribute__((aligned(16))) char dyn[];
  __shared__ RowShared sh;
  uint64_t* keys = reinterpret_cast<uint64_t*>(dyn);                          // [cap] candidates
  uint4* hit = reinterpret_cast<uint4*>(dyn + (size_t)a.cap * 8);             // [hits] vectors reaching tau
  int32_t* hit_v = reinterpret_cast<int32_t*>(dyn + (size_t)a.cap * 8 + (size_t)a.hits * 16);
  const int o = (int)(blockIdx.x / (unsigned)a.nseg), seg = (int)(blockIdx.x - (unsigned)o * a.nseg);
  int i, k;
  if (!live_row(sh.live, o, a.B, a.G, a.lengths, a.temperature, i, k)) return;   // the merge kernel fills the other rows
  const int r = i * a.G + k;
  const float T = a.temperature[i];
  const char* row = reinterpret_cast<const char*>(a.target) + ((size_t)i * (a.G + 1) + k) * (size_t)a.V * Seg::ES;
  const Seg g(row, a.V, seg, a.nseg);
  uint4 d[kSegVecs];
  g.load(row, d);
  const float x = g.load_scalar(row);
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  if (tid == 0) sh.n = sh.nhit = 0;

  float zm = x;   // the lane's largest value so far
  uint32_t tau = kNegInfKey;
  float tz = -INFINITY;
  // waves whose lanes all hold a vector of the segment
  const int full = min((g.ve - g.vb) >> 6, kSegWaves);
  const int need = full ? (a.K + full - 1) / full : SPEC_WAVE + 1;
  int turn = 0;
  auto raise_tau = [&]() {
    // the wave's need-th largest lane maximum, bitwise from the top: bf16 keys end at bit 16, and a bound on
    // fp32 keys need not go below bit 14
    const uint32_t key = order_key(zm);
    uint32_t t = need > SPEC_WAVE ? kNegInfKey : 0xffffffffu;
    if (wave < full && need <= SPEC_WAVE) {
      t = 0;
#pragma unroll
      for (int bit = 31; bit >= (BF16 ? 16 : 14); --bit) {
        const uint32_t trial = t | (1u << bit);
        if ((int)__popcll(__ballot(key >= trial)) >= need) t = trial;
      }
      if (BF16 && t < 0x80000000u) t |= 0xffffu;
      t = max(t, kNegInfKey);
    }
    if (lane == 0) sh.t[turn][wave] = t;
    lds_barrier();   // one turn's values are read before the next turn's barrier, and written anew behind it
    tau = sh.t[turn][0];
#pragma unroll
    for (int w = 1; w < kSegWaves; ++w) tau = min(tau, sh.t[turn][w]);
    tz = key_value(tau);
    turn ^= 1;
  };
  auto largest = [&](const float (&z)[EPV]) {
    float m = z[0];
#pragma unroll
    for (int e = 1; e < EPV; ++e) m = fmaxf(m, z[e]);
    return m;
  };
  // the first bound, from the first chunk's maxima (it stays in registers)
#pragma unroll
  for (int j = 0; j < kSegVecs; ++j) {
    float z[EPV];
    Seg::unpack(d[j], z);
    if (g.vb + j * kSegThreads + tid < g.ve) zm = fmaxf(zm, largest(z));
    asm volatile("" : "+v"(zm));
  }
  forget(d);
  float S = 0.f;
  const Reference rf = pick_reference(sh.sum, zm, T);
  raise_tau();
  int chunk = 0;
#pragma unroll 1
  for (int c = g.vb; c < g.ve; c += kSegChunk) {
    g.walk_chunk(row, c, d, [&](int v, const uint4& q) {
      float z[EPV];
      Seg::unpack(q, z);
      S += exp_sum<EPV>(z, rf.c_f, rf.M);
      const float m = largest(z);
      zm = fmaxf(zm, m);
      if (m >= tz && m > -INFINITY) {   // copied whole; its values are looked at one by one below
        const int h = atomicAdd(&sh.nhit, 1);
        if (h < a.hits) {
          hit[h] = q;
          hit_v[h] = v;
        }
      }
      asm volatile("" : "+v"(S));   // one vector's values at a time: registers
    });
    ++chunk;
    // (at the end only for long lists: it halves the candidates)
    if (chunk > 1 && (c + kSegChunk < g.ve ? (chunk & (chunk - 1)) == 0 : a.K > SPEC_WAVE)) raise_tau();
  }
  if (g.nx > 0) {
    const float z1[1] = {x};
    S += exp_sum<1>(z1, rf.c_f, rf.M);
  }
  const uint4* body = reinterpret_cast<const uint4*>(row + (size_t)g.head * Seg::ES);
  int bad;
  const SegSum total =
      segment_sum<BF16>(sh.sum, S, rf, T, g, [&](int v) { return body[v]; }, x, bad);
  __syncthreads();
  // the candidates: values that reach the last tau
  const int nhit = sh.nhit;
  auto list = [&](float z, int id) {
    if (z >= tz && z > -INFINITY) {
      const int s = atomicAdd(&sh.n, 1);
      if (s < a.cap) keys[s] = pack_key(z, id);
    }
  };
  if (nhit <= a.hits) {
    for (int h = tid; h < nhit; h += kSegThreads) {
      float z[EPV];
      Seg::unpack(hit[h], z);
      const int v = hit_v[h];
#pragma unroll
      for (int e = 0; e < EPV; ++e) list(z[e], g.id_of(v, e));
    }
    if (tid < g.nx) list(x, g.id_of_scalar(tid));
  }
  __syncthreads();
  int n = sh.n;
  if (n > a.cap || nhit > a.hits) {
    // more than `cap` values reach tau: the K-th key exactly, counting over the segment again
    int step = 0;
    auto count = [&](auto pred) -> int {
      int c = tid < g.nx && pred(order_key(x + 0.f), g.id_of_scalar(tid)) ? 1 : 0;
#pragma unroll 1
      for (int v = g.vb + tid; v < g.ve; v += kSegThreads) {
        float z[EPV];
        Seg::unpack(body[v], z);
#pragma unroll
        for (int e = 0; e < EPV; ++e) c += pred(order_key(z[e] + 0.f), g.id_of(v, e)) ? 1 : 0;
      }
      c = wave_sum_i(c);
      if (lane == 0) sh.sel.cnt[step & 1][wave] = c;
      __syncthreads();
      int tot = 0;
#pragma unroll
      for (int w = 0; w < kSegWaves; ++w) tot += sh.sel.cnt[step & 1][w];
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
        if (s < a.cap) keys[s] = pack_key(z, id);
      }
    };
#pragma unroll 1
    for (int v = g.vb + tid; v < g.ve; v += kSegThreads) {
      float z[EPV];
      Seg::unpack(body[v], z);
#pragma unroll
      for (int e = 0; e < EPV; ++e) take(z[e], g.id_of(v, e));
    }
    if (tid < g.nx) take(x, g.id_of_scalar(tid));
    __syncthreads();
    n = min(sh.n, a.cap);
    tau = th;
  }
  if (a.nseg > 1) {
    uint64_t* out = a.keys + ((size_t)r * a.nseg + seg) * a.cap;
    for (int e = tid; e < n; e += kSegThreads) out[e] = keys[e];
  } else {
    if (tid < SPEC_WAVE) select_topk<BF16 ? 16 : 0>(sh.sel, keys, n, a.K, tau);
    __syncthreads();
    write_list<kSegWaves>(sh.sel, a, r);
    if (a.lse && tid == 0) a.lse[r] = (float)(0.69314718055994530942 * (total.ref + log2(total.sum)));
  }
  if (tid == 0) a.segs[(size_t)r * a.nseg + seg] = TeacherSeg{total.sum, total.ref, bad, tau, n, 0};
}

constexpr int kMergeThreads = 256;

template <int SH>
__global__ __launch_bounds__(kMergeThreads) void teacher_merge_kernel(TeacherArgs a) {
  __shared__ SelectShared sel;
  __shared__ uint64_t keys[kMergeKeys];
  __shared__ int sbad, sn;
  const int r = (int)blockIdx.x, i = r / a.G, k = r - i * a.G, tid = threadIdx.x;
  const int L = a.lengths ? a.lengths[i] : a.G;
  const float T = a.temperature[i];
  int st = 0;
  if (L < 0 || L > a.G) {
    st = SPEC_REQ_BAD_LENGTH;
  } else if (!(T > 0.f && T < INFINITY)) {
    st = SPEC_REQ_BAD_TEMPERATURE;
  } else if (L > 0) {
    // every row of the request: a bad or an empty one marks the request
    if (tid == 0) sbad = 0;
    __syncthreads();
    if (tid < L) {
      const TeacherSeg* q = a.segs + ((size_t)i * a.G + tid) * a.nseg;
      int bad = 0, some = 0;
      for (int s = 0; s < a.nseg; ++s) {
        bad |= q[s].bad;
        some |= q[s].sum > 0.0;
      }
      if (bad || !some) sbad = 1;
    }
    __syncthreads();
    if (sbad) st = SPEC_REQ_NONFINITE;
  }
  if (a.status && k == 0 && tid == 0) a.status[i] = st;
  if (st != 0 || k >= L) {
    write_empty(a, r, st != 0 ? NAN : -INFINITY);
    return;
  }
  if (a.nseg == 1) return;   // written by the row's own workgroup
  const TeacherSeg* p = a.segs + (size_t)r * a.nseg;
  uint32_t tau = kNegInfKey;
  for (int s = 0; s < a.nseg; ++s) tau = max(tau, p[s].tau);
  int cur = 0, s0 = 0;
  while (s0 < a.nseg) {   // rounds: the keys kept so far and as many segments' lists as fit
    if (tid == 0) sn = cur;
    for (int e = tid; e < cur; e += (int)blockDim.x) keys[e] = sel.list[e];
    __syncthreads();
    int total = cur, s1 = s0;
    while (s1 < a.nseg && total + p[s1].n <= kMergeKeys) total += p[s1++].n;
    for (int s = s0; s < s1; ++s) {
      const uint64_t* src = a.keys + ((size_t)r * a.nseg + s) * a.cap;
      for (int e = tid; e < p[s].n; e += kMergeThreads) {
        const uint64_t key = src[e];
        if ((uint32_t)(key >> 32) >= tau) keys[atomicAdd(&sn, 1)] = key;
      }
    }
    __syncthreads();
    if (tid < SPEC_WAVE) select_topk<SH>(sel, keys, sn, a.K, tau);
    __syncthreads();
    cur = sel.n;
    s0 = s1;
  }
  write_list<kMergeThreads / SPEC_WAVE>(sel, a, r);
  if (a.lse && tid == 0) {
    double ref = -INFINITY, S = 0.0;
    for (int s = 0; s < a.nseg; ++s)
      if (p[s].sum > 0.0) ref = fmax(ref, p[s].ref);
    for (int s = 0; s < a.nseg; ++s)
      if (p[s].sum > 0.0) S += p[s].sum * exp2(p[s].ref - ref);
    a.lse[r] = (float)(0.69314718055994530942 * (ref + log2(S)));
  }
}

// Candidates a segment of at most `vecs` vectors of EPV values may list: on Gaussian rows 22 (K = 1) to 460
// (K = 256) reach tau on average, 700 at most seen of 160 segments.  Where the full waves are too few to take
// tau from (more than 64 values of each: a row of fewer than 258 vectors), everything is listed.  (By the first
// rule alone they took the 53 counting passes of tied rows: 256 x 16 of 1500 bf16, K = 200: 281 us in place of 197.)
constexpr int least_waves(int vecs) { return vecs < 66 ? 0 : vecs >= 514 ? kSegWaves : (vecs - 2) >> 6; }
constexpr bool no_bound(int vecs, int K) { return K > SPEC_WAVE * least_waves(vecs); }
constexpr int list_cap(int vecs, int epv, int K) {   // even: the vectors behind the keys lie on 16 bytes
  const int some = 3 * K + 640 + (K & 1), all = vecs * epv + 14;
  return no_bound(vecs, K) && all > some ? all + (all & 1) : some;
}
// Vectors reaching one of the earlier bounds: one such lot per doubling, and each vector once at most.
constexpr int hit_cap(int vecs, int K) { return vecs < 6 * K + 288 ? vecs + 1 : 6 * K + 288; }

constexpr bool lists_fit() {
  for (int epv : {4, 8})
    for (int K : {1, 64, 65, 128, 129, 192, 193, 256})
      for (int vecs = 0; vecs < 700; ++vecs)
        // a segment of vecs or up to two fewer vectors, and 14 scalars, without a bound
        if (K > SPEC_WAVE * (vecs < 66 ? 0 : (vecs - 2) / SPEC_WAVE) && vecs * epv + 14 > list_cap(vecs, epv, K)) return false;
  return true;
}
static_assert(lists_fit(), "a segment that has no bound lists all of its values");
static_assert(!no_bound(kSegChunk / 2, SPEC_MAX_TEACHER_K), "segments of a row cut into several have a bound");
static_assert(3 * SPEC_MAX_TEACHER_K + 641 + SPEC_MAX_TEACHER_K <= kMergeKeys, "a list fits a round of the merge");

// Vectors of a segment at most.
int segment_vecs(int V, int dtype, int nseg) { return (V / (dtype == SPEC_BF16 ? 8 : 4) + nseg - 1) / nseg; }

size_t segs_bytes(size_t rows, int nseg) { return round256(rows * nseg * sizeof(TeacherSeg)); }
size_t keys_bytes(size_t rows, int nseg, int cap) {
  return nseg > 1 ? round256(rows * nseg * (size_t)cap * sizeof(uint64_t)) : 0;
}
int teacher_cap(int V, int dtype, int nseg, int K) {
  return list_cap(segment_vecs(V, dtype, nseg), dtype == SPEC_BF16 ? 8 : 4, K);
}

}  // namespace
}  // namespace spec

using namespace spec;

extern "C" size_t spec_teacher_workspace_size(int32_t B, int32_t gamma, int32_t V, int32_t K) {
  if (!shape_ok(B, gamma, V, SPEC_BF16) || K < 1 || K > SPEC_MAX_TEACHER_K) return 0;
  const size_t rows = (size_t)B * gamma;
  size_t most = 0;
  for (int dtype : {SPEC_F32, SPEC_BF16}) {   // the larger of the two storage types'
    const int nseg = row_segments((int64_t)rows, V, dtype);
    const size_t n = segs_bytes(rows, nseg) + keys_bytes(rows, nseg, teacher_cap(V, dtype, nseg, K));
    if (n > most) most = n;
  }
  return most;
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
  const uint64_t rows = (uint64_t)B * gamma;
  a.nseg = row_segments((int64_t)rows, V, dtype);
  a.cap = teacher_cap(V, dtype, a.nseg, K);
  a.hits = hit_cap(segment_vecs(V, dtype, a.nseg), K);
  if (rows * a.nseg * kSegThreads > 0xffffffffull) return SPEC_ERR_UNSUPPORTED;
  a.target = target_logits; a.lengths = lengths; a.temperature = temperature;
  a.ids = ids_out; a.values = values_out; a.lse = lse_out; a.status = status;
  a.segs = reinterpret_cast<TeacherSeg*>(workspace);
  a.keys = reinterpret_cast<uint64_t*>(reinterpret_cast<char*>(workspace) + segs_bytes(rows, a.nseg));
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  const dim3 grid((unsigned)(rows * a.nseg));
  const unsigned lds = (unsigned)(a.cap * 8 + a.hits * 20);
  if (dtype == SPEC_BF16) {
    hipLaunchKernelGGL(teacher_row_kernel<true>, grid, dim3(kSegThreads), lds, s, a);
    hipLaunchKernelGGL(teacher_merge_kernel<16>, dim3((unsigned)rows), dim3(kMergeThreads), 0, s, a);
  } else {
    hipLaunchKernelGGL(teacher_row_kernel<false>, grid, dim3(kSegThreads), lds, s, a);
    hipLaunchKernelGGL(teacher_merge_kernel<0>, dim3((unsigned)rows), dim3(kMergeThreads), 0, s, a);
  }
  return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_ERR_HIP;
}
