// Penalties, biases and masks on logits, row by row of a draft block, on gfx950.
//
//   count of row k = the token's occurrences in the request's output and in the draft tokens before row k
//   z = z > 0 ? z / repetition : z * repetition   (a token of the prompt, or of count > 0)
//   z = z - frequency * count;  z = z - presence (count > 0);  z = z + bias;  z = -inf where the mask's bit is 0
//
// Nearly all of a row stays as it is: a history names a few thousand tokens of the vocabulary.  Workgroups count the
// history's tokens in LDS (a word per token; the first to count a token puts it on a list) and then go through the
// block's rows, which share one count; the draft tokens before a row are compared with the listed token one by one.
//   Out of place, under a mask, or where much may be listed: a workgroup takes a request and a slice of the
//   vocabulary.  The slice of a row goes through LDS, where lanes take the listed tokens (adjusted in the registers
//   that carry the rows, a lane here and there of every wave, it took as long as the copy itself).  Masks are applied on
//   the way out.  In place, pieces without a count are written only where the mask forbids a value, and read only where
//   it forbids some.
//   In place without a mask and with few tokens: a workgroup takes a request and a class of its tokens, found through a
//   hash table; lanes take pairs of listed token and row in memory.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <utility>

#include "adjust_plan.hpp"
#include "common.hpp"
#include "rowseg.hpp"
#include "spec_verify.h"

namespace spec {
namespace {

constexpr int kProbes = 64;
constexpr uint32_t kInPrompt = 1u << 30, kDrafted = 1u << 31, kBiased = 1u << 29, kCount = kBiased - 1;

struct AdjustArgs {
  const char* logits;   // [B, R, V]
  char* out;
  const int32_t* draft_tokens;   // [B, gamma]
  const int32_t* lengths;
  const int32_t* history;        // [B, H]
  const int32_t* history_len;
  const int32_t* prompt_len;
  const float* repetition;
  const float* frequency;
  const float* presence;
  const int32_t* bias_offsets;   // [B + 1]
  const int32_t* bias_tokens;
  const float* bias_values;
  const uint32_t* mask;          // [masks, R, words]
  const int32_t* mask_index;
  int32_t* status;
  int R, V, gamma, H, bias_count, masks, words;
};

// 16 bytes of a row; rows start on no boundary where V is odd.
template <int ALIGN>
struct __attribute__((packed, aligned(ALIGN))) Piece {
  v4u32 v;
};

template <bool BF16>
__device__ __forceinline__ void store_elem(char* row, int64_t v, float z) {
  if constexpr (BF16) reinterpret_cast<__bf16*>(row)[v] = (__bf16)z;
  else reinterpret_cast<float*>(row)[v] = z;
}

// A request's own numbers; every workgroup of the request comes to the same verdict.
struct Request {
  int st = 0, live, hl, pl, need, bo = 0, bn = 0, mi;
  float rep, freq, pres;
  bool penal;   // else neither history nor drafts matter
};

template <bool BIAS>
__device__ __forceinline__ Request request(const AdjustArgs& a, int b) {
  Request q;
  const int L = a.lengths ? a.lengths[b] : a.gamma;
  if (L < 0 || L > a.gamma) q.st |= SPEC_REQ_BAD_LENGTH;
  q.live = q.st ? 0 : L + (a.R - a.gamma);
  q.hl = a.history ? (a.history_len ? a.history_len[b] : a.H) : 0;
  q.pl = a.history && a.prompt_len ? a.prompt_len[b] : 0;
  if (q.hl < 0 || q.hl > a.H || q.pl < 0 || q.pl > q.hl) {
    q.st |= SPEC_REQ_BAD_LENGTH;
    q.hl = q.pl = 0;
  }
  q.rep = a.repetition ? a.repetition[b] : 1.f;
  q.freq = a.frequency ? a.frequency[b] : 0.f;
  q.pres = a.presence ? a.presence[b] : 0.f;
  if (!(q.rep > 0.f && q.rep < INFINITY && fabsf(q.freq) < INFINITY && fabsf(q.pres) < INFINITY))
    q.st |= SPEC_REQ_BAD_PENALTY;
  q.penal = q.rep != 1.f || q.freq != 0.f || q.pres != 0.f;
  if constexpr (BIAS) {
    q.bo = a.bias_offsets[b];
    const int be = a.bias_offsets[b + 1];
    if (q.bo < 0 || be < q.bo || be > a.bias_count) q.st |= SPEC_REQ_BAD_LIST;
    else q.bn = be - q.bo;
  }
  q.mi = a.mask ? (a.mask_index ? a.mask_index[b] : b) : -1;
  if (q.mi < -1 || q.mi >= a.masks) q.st |= SPEC_REQ_BAD_MASK;
  q.need = q.penal ? min(q.live - 1, a.gamma) : 0;   // draft tokens that precede a live row
  return q;
}

// What a request's rows count and add, put into a workgroup's tables: slot_of names a token's slot (past `slots`:
// none).  `note` is told the slot and what its count was.  Returns whether a token is out of range.
template <bool BIAS, int T, class Slot, class Note>
__device__ __forceinline__ bool gather(const AdjustArgs& a, const Request& q, int b, const int32_t* drafts, uint32_t* count,
                                       uint32_t* bias_at, unsigned slots, Slot slot_of, Note note) {
  const int tid = threadIdx.x;
  bool off = false;
  if (q.penal && q.live > 0) {
    const int32_t* h = a.history + (size_t)b * a.H;
    // four tokens a load, F loads in flight per thread
    constexpr int F = 4;
    const int quads = q.hl >> 2;
    uint32_t most = 0;   // of t + 1: -1 is a hole
    auto count_in = [&](int t, int i) {
      most = max(most, (unsigned)t + 1u);
      const unsigned at = slot_of(t);
      if (at < slots) note(at, t, i < q.pl ? atomicOr(&count[at], kInPrompt) : atomicAdd(&count[at], 1u));
    };
    for (int i0 = tid; i0 < quads; i0 += F * T) {
      v4u32 t[F];
#pragma unroll
      for (int u = 0; u < F; ++u) {
        t[u] = v4u32{~0u, ~0u, ~0u, ~0u};
        if (i0 + u * T < quads) t[u] = reinterpret_cast<const Piece<4>*>(h + 4 * (i0 + u * T))->v;
      }
#pragma unroll
      for (int u = 0; u < F; ++u)
#pragma unroll
        for (int x = 0; x < 4; ++x) count_in((int)t[u][x], 4 * (i0 + u * T) + x);
    }
    if (tid < (q.hl & 3)) count_in(h[4 * quads + tid], 4 * quads + tid);
    off |= most > (unsigned)a.V;
    if (tid < q.need) {
      const int t = drafts[tid];
      const unsigned at = slot_of(t);
      off |= (unsigned)t >= (unsigned)a.V;
      if (at < slots) note(at, t, atomicOr(&count[at], kDrafted));
    }
  }
  if constexpr (BIAS) {
    // unsigned: the step behind the last entry may pass 2^31
    for (unsigned i = tid; i < (unsigned)q.bn && q.live > 0; i += T) {
      const int t = a.bias_tokens[(unsigned)q.bo + i];
      const unsigned at = slot_of(t);
      off |= (unsigned)t >= (unsigned)a.V;
      if (at < slots) {
        note(at, t, atomicOr(&count[at], kBiased));
        atomicMax(&bias_at[at], i + 1);
      }
    }
  }
  return off;
}

// A listed token: what is the same for every row.
struct Token {
  int id, c;
  bool prompt, drafted, biased;
  float bias;
};

template <bool BIAS>
__device__ __forceinline__ Token token(const AdjustArgs& a, const Request& q, int id, uint32_t w, const uint32_t* bias_at, int at) {
  Token t{id, (int)(w & kCount), (w & kInPrompt) != 0, (w & kDrafted) != 0, BIAS && (w & kBiased), 0.f};
  if constexpr (BIAS)
    if (t.biased) t.bias = a.bias_values[q.bo + (int)bias_at[at] - 1];
  return t;
}

__device__ __forceinline__ float adjusted(const Request& q, const int32_t* drafts, float z, const Token& t, int r) {
  int c = t.c;
  if (t.drafted)
    for (int k = 0; k < min(r, q.need); ++k) c += drafts[k] == t.id;
  if (c > 0 || t.prompt) z = z > 0.f ? z / q.rep : z * q.rep;
  if (c > 0) {
    z = z - q.freq * (float)c;
    z = z - q.pres;
  }
  if (t.biased) z = z + t.bias;
  return z;
}

// S tokens of the vocabulary and T threads per workgroup.
template <bool BF16, bool BIAS, bool COPY, int S, int T>
__global__ __launch_bounds__(T) void adjust_kernel(AdjustArgs a) {
  constexpr int ES = BF16 ? 2 : 4, VE = 16 / ES, NV = S / VE / T;   // pieces of a row per lane
  static_assert(S % (VE * T) == 0 && S <= 65536, "slice");
  __shared__ __attribute__((aligned(16))) uint32_t count[S];
  __shared__ __attribute__((aligned(16))) uint32_t bias_at[BIAS ? S : 4];   // entry of the list + 1 (the last one of a token named twice)
  __shared__ __attribute__((aligned(16))) char part[S * ES];
  __shared__ uint16_t list[S];
  __shared__ int32_t drafts[SPEC_MAX_GAMMA];
  __shared__ int listed, bad;
  const int tid = threadIdx.x, V = a.V, R = a.R, slices = (V + S - 1) / S;
  const int b = (int)(blockIdx.x / (unsigned)slices), slice = (int)(blockIdx.x % (unsigned)slices);
  const int v0 = slice * S, n = min(S, V - v0);
  const Request q = request<BIAS>(a, b);
  int st = q.st;

  // row r's allowed values of the lane's pieces (0 where there is none)
  constexpr uint32_t kAll = (1u << VE) - 1;
  const uint32_t* mask = q.mi >= 0 && !q.st ? a.mask + (size_t)q.mi * R * a.words : nullptr;
  const size_t row0 = (size_t)b * R * V + v0;
  uint32_t some[NV] = {};   // in place: a lane's values with a count
  auto load_on = [&](int r, uint32_t(&on)[NV]) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = (tid + k * T) * VE, left = n - i;
      on[k] = left >= VE ? kAll : left > 0 ? (1u << left) - 1 : 0u;
      if (mask && left > 0) on[k] &= mask[(size_t)r * a.words + ((v0 + i) >> 5)] >> ((v0 + i) & 31);
    }
  };
  // in place only what changes is read: a value with a count, or one beside a forbidden one
  auto moves = [&](int k, uint32_t on) {
    const int i = (tid + k * T) * VE;
    const uint32_t whole = i + VE <= n ? kAll : (1u << max(n - i, 0)) - 1;
    return COPY ? on != 0 : (on & some[k]) != 0 || (on != 0 && on != whole);
  };
  auto load_row = [&](int r, const uint32_t(&on)[NV], v4u32(&z)[NV]) {
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = (tid + k * T) * VE;
      if (!moves(k, on[k])) continue;
      const size_t at = row0 + (size_t)r * V + i;
      if (i + VE <= n) {
        z[k] = __builtin_nontemporal_load(&reinterpret_cast<const Piece<ES>*>(a.logits + at * ES)->v);
      } else {   // the row's last values
        z[k] = v4u32{};
        for (int x = 0; i + x < n; ++x) {
          const uint32_t h = BF16 ? reinterpret_cast<const uint16_t*>(a.logits)[at + x] : reinterpret_cast<const uint32_t*>(a.logits)[at + x];
          if constexpr (BF16) {
            if (x < 2) z[k].x |= h << (16 * x);
            else if (x < 4) z[k].y |= h << (16 * (x - 2));
            else if (x < 6) z[k].z |= h << (16 * (x - 4));
            else z[k].w |= h << (16 * (x - 6));
          } else {
            if (x == 0) z[k].x = h;
            else if (x == 1) z[k].y = h;
            else z[k].z = h;
          }
        }
      }
    }
  };
  uint32_t next_on[NV] = {};
  v4u32 next[NV] = {};
  // the first row comes while the history is counted, the others while the one before is adjusted (90 -> 83 us)
  if (COPY && q.live > 0) {
    load_on(0, next_on);
    load_row(0, next_on, next);
  }

  for (int i = tid; i < S / 4; i += T) {
    reinterpret_cast<v4u32*>(count)[i] = v4u32{};
    if constexpr (BIAS) reinterpret_cast<v4u32*>(bias_at)[i] = v4u32{};
  }
  if (tid == 0) listed = bad = 0;
  if (tid < q.need) drafts[tid] = a.draft_tokens[(size_t)b * a.gamma + tid];
  __syncthreads();
  if (gather<BIAS, T>(a, q, b, drafts, count, bias_at, (unsigned)n, [&](int t) { return (unsigned)t - (unsigned)v0; },
                      [&](unsigned at, int, uint32_t old) {
                        if (old == 0) list[atomicAdd(&listed, 1)] = (uint16_t)at;
                      }))
    bad = 1;
  __syncthreads();
  if (bad) st |= SPEC_REQ_BAD_TOKEN;
  if (slice == 0 && tid == 0 && a.status) a.status[b] = st;
  if (st || q.live == 0) return;

  const int E = listed, live = q.live;
  auto entry = [&](int e) { return token<BIAS>(a, q, v0 + list[e], count[list[e]], bias_at, list[e]); };

  if (!COPY) {
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int x = 0; x < VE; ++x) some[k] |= (count[(tid + k * T) * VE + x] ? 1u : 0u) << x;
    load_on(0, next_on);
    load_row(0, next_on, next);
  }
  Token mine{};   // the lane's first listed token
  if (tid < E) mine = entry(tid);
  for (int r = 0; r < live; ++r) {
    v4u32 z[NV];
    uint32_t on[NV];
    bool move[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      z[k] = next[k];
      on[k] = next_on[k];
      move[k] = moves(k, on[k]);
    }
    if (r + 1 < live) {
      load_on(r + 1, next_on);
      load_row(r + 1, next_on, next);
    }
    if (E > 0) {
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (move[k]) *reinterpret_cast<v4u32*>(&part[(tid + k * T) * 16]) = z[k];
      __syncthreads();
      for (int e = tid; e < E; e += T) {
        const Token t = e == tid ? mine : entry(e);
        store_elem<BF16>(part, t.id - v0, adjusted(q, drafts, load_elem<BF16>(part, t.id - v0), t, r));
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < NV; ++k)
        if (move[k]) z[k] = *reinterpret_cast<const v4u32*>(&part[(tid + k * T) * 16]);
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int i = (tid + k * T) * VE;
      if (i >= n || (!COPY && !move[k] && on[k] != 0)) continue;
      const size_t at = row0 + (size_t)r * V + i;
      v4u32 y = move[k] ? z[k] : v4u32{};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        if constexpr (BF16) {
          const uint32_t p = on[k] >> (2 * x) & 3u, keep = (p & 1u ? 0xffffu : 0u) | (p & 2u ? 0xffff0000u : 0u);
          y[x] = (y[x] & keep) | (0xff80ff80u & ~keep);
        } else {
          y[x] = on[k] >> x & 1u ? y[x] : 0xff800000u;
        }
      }
      if (i + VE <= n) {
        __builtin_nontemporal_store(y, &reinterpret_cast<Piece<ES>*>(a.out + at * ES)->v);
      } else {
#pragma unroll
        for (int x = 0; x < VE; ++x) {
          if (i + x >= n) break;
          if constexpr (BF16) reinterpret_cast<uint16_t*>(a.out)[at + x] = (uint16_t)(y[x / 2] >> (x & 1 ? 16 : 0));
          else reinterpret_cast<uint32_t*>(a.out)[at + x] = y[x];
        }
      }
    }
  }
}

// In place and without a mask: the listed tokens alone, where they lie.  A workgroup takes the tokens of a class, every
// 2^bits-th block of 64 (lines of memory belong to one class), counts them in a table of kSlots that a token's hash
// leads into, and its lanes take pairs of listed token and row.  A class of more tokens than the table takes is gone
// through again, kSlots of the class at a time, in order.
template <bool BF16, bool BIAS>
__global__ __launch_bounds__(kFewThreads) void adjust_few_kernel(AdjustArgs a, int bits) {
  constexpr int T = kFewThreads, U = 4;   // pairs in flight per lane
  __shared__ int32_t key[kSlots];
  __shared__ uint32_t count[kSlots];
  __shared__ uint32_t bias_at[BIAS ? kSlots : 1];
  __shared__ uint16_t list[kSlots];
  __shared__ int32_t drafts[SPEC_MAX_GAMMA];
  __shared__ int listed, bad, over;
  const int tid = threadIdx.x, V = a.V, R = a.R;
  const int classes = 1 << bits, b = (int)(blockIdx.x >> bits), mine = (int)blockIdx.x & (classes - 1);
  const Request q = request<BIAS>(a, b);
  int st = q.st;
  auto clear = [&] {
    for (int i = tid; i < kSlots; i += T) {
      key[i] = -1;
      count[i] = 0;
      if constexpr (BIAS) bias_at[i] = 0;
    }
    if (tid == 0) listed = 0;
  };
  auto in_class = [&](int t) { return (unsigned)t < (unsigned)V && ((t >> 6) & (classes - 1)) == mine; };
  const size_t row0 = (size_t)b * R * V;
  auto entry = [&](int e) { return token<BIAS>(a, q, key[list[e]], count[list[e]], bias_at, list[e]); };
  auto write = [&] {
    const unsigned E = (unsigned)listed, pairs = E * (unsigned)q.live;
    for (unsigned p0 = tid; p0 < pairs; p0 += U * T) {
      float z[U];
      Token t[U];
      int r[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const unsigned p = min(p0 + u * T, pairs - 1);
        r[u] = (int)(p / E);
        t[u] = entry((int)(p % E));
        z[u] = load_elem<BF16>(a.logits, (int64_t)(row0 + (size_t)r[u] * V + t[u].id));
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (p0 + u * T < pairs)
          store_elem<BF16>(a.out, (int64_t)(row0 + (size_t)r[u] * V + t[u].id), adjusted(q, drafts, z[u], t[u], r[u]));
    }
  };

  clear();
  if (tid == 0) bad = over = 0;
  if (tid < q.need) drafts[tid] = a.draft_tokens[(size_t)b * a.gamma + tid];
  __syncthreads();
  if (gather<BIAS, T>(a, q, b, drafts, count, bias_at, (unsigned)kSlots,
                      [&](int t) {
                        if (!in_class(t)) return ~0u;
                        unsigned at = (unsigned)t * 2654435761u >> (32 - kSlotBits);
                        for (int probe = 0; probe < kProbes; ++probe, at = (at + 1) & (kSlots - 1)) {
                          const int old = atomicCAS(&key[at], -1, t);
                          if (old == -1 || old == t) return at;
                        }
                        over = 1;
                        return ~0u;
                      },
                      [&](unsigned at, int, uint32_t old) {
                        if (old == 0) list[atomicAdd(&listed, 1)] = (uint16_t)at;
                      }))
    bad = 1;
  __syncthreads();
  if (bad) st |= SPEC_REQ_BAD_TOKEN;
  if (mine == 0 && tid == 0 && a.status) a.status[b] = st;
  if (st) return;
  if (!over) {
    write();
    return;
  }
  for (int c0 = 0; c0 < ((V - 1) >> (6 + bits) << 6) + 64; c0 += kSlots) {
    __syncthreads();   // the table is read no more
    clear();
    __syncthreads();
    gather<BIAS, T>(a, q, b, drafts, count, bias_at, (unsigned)kSlots,
                    [&](int t) { return in_class(t) ? (unsigned)((t >> (6 + bits) << 6 | (t & 63)) - c0) : ~0u; },
                    [&](unsigned at, int t, uint32_t old) {
                      if (old == 0) {
                        key[at] = t;
                        list[atomicAdd(&listed, 1)] = (uint16_t)at;
                      }
                    });
    __syncthreads();
    write();
  }
}

template <bool BF16, bool BIAS, bool COPY, int S, int T>
void launch(const AdjustArgs& a, dim3 grid, hipStream_t s) {
  hipLaunchKernelGGL((adjust_kernel<BF16, BIAS, COPY, S, T>), grid, dim3(T), 0, s, a);
}

template <bool BF16, bool BIAS>
void run_adjust(const AdjustArgs& a, int B, const AdjustPlan& p, hipStream_t s) {
  const bool copy = a.logits != a.out;
  const dim3 grid((unsigned)p.workgroups(B, a.V));
  if (p.bits >= 0) {
    hipLaunchKernelGGL((adjust_few_kernel<BF16, BIAS>), grid, dim3(kFewThreads), 0, s, a, p.bits);
    return;
  }
  if constexpr (BF16 && !BIAS) {
    if (p.slice == 2 * kSlice) {
      if (copy) launch<BF16, BIAS, true, 2 * kSlice, 1024>(a, grid, s);
      else launch<BF16, BIAS, false, 2 * kSlice, 1024>(a, grid, s);
      return;
    }
  }
  if (copy) launch<BF16, BIAS, true, kSlice, slice_threads(BF16)>(a, grid, s);
  else launch<BF16, BIAS, false, kSlice, slice_threads(BF16)>(a, grid, s);
}

}  // namespace
}  // namespace spec

using namespace spec;

extern "C" int32_t spec_adjust_logits(int32_t B, int32_t R, int32_t V, int32_t dtype, const void* logits, int32_t gamma,
                                      const int32_t* draft_tokens, const int32_t* lengths, const int32_t* history,
                                      int32_t H, const int32_t* history_len, const int32_t* prompt_len,
                                      const float* repetition, const float* frequency, const float* presence,
                                      const int32_t* bias_offsets, const int32_t* bias_tokens, const float* bias_values,
                                      int32_t bias_count, const uint32_t* mask, int32_t masks, const int32_t* mask_index,
                                      void* logits_out, int32_t* status, void* stream) {
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_ERR_INVALID_ARG;
  if (B < 1 || gamma < 0 || gamma > SPEC_MAX_GAMMA || R < 1 || (R != gamma && R != gamma + 1)) return SPEC_ERR_INVALID_ARG;
  if (V < 1 || V > (dtype == SPEC_BF16 ? SPEC_MAX_V : SPEC_MAX_V / 2)) return SPEC_ERR_INVALID_ARG;
  if (!logits || !logits_out || !aligned16(logits) || !aligned16(logits_out)) return SPEC_ERR_INVALID_ARG;
  if (gamma > 0 && !draft_tokens) return SPEC_ERR_INVALID_ARG;
  if (history ? H < 1 || H > SPEC_MAX_HISTORY : H != 0 || history_len || prompt_len) return SPEC_ERR_INVALID_ARG;
  if (!bias_offsets != !bias_tokens || !bias_offsets != !bias_values || bias_count < 0 || (!bias_offsets && bias_count))
    return SPEC_ERR_INVALID_ARG;
  if (mask ? masks < 1 || (!mask_index && masks < B) : masks != 0 || mask_index) return SPEC_ERR_INVALID_ARG;
  const size_t bytes = (size_t)B * R * V * (dtype == SPEC_BF16 ? 2 : 4), words = (size_t)ceil_div(V, 32);
  if (logits_out != logits && overlap(logits_out, bytes, logits, bytes)) return SPEC_ERR_INVALID_ARG;
  const size_t per = (size_t)B * sizeof(int32_t), nb = (size_t)bias_count * sizeof(int32_t);
  for (auto [p, m] : {std::pair<const void*, size_t>{draft_tokens, per * gamma}, {lengths, per}, {history, per * H},
                      {history_len, per}, {prompt_len, per}, {repetition, per}, {frequency, per}, {presence, per},
                      {bias_offsets, per + sizeof(int32_t)}, {bias_tokens, nb}, {bias_values, nb},
                      {mask, (size_t)masks * R * words * sizeof(uint32_t)}, {mask_index, per}})
    if (overlap(logits_out, bytes, p, m) || overlap(status, per, p, m)) return SPEC_ERR_INVALID_ARG;
  if (overlap(status, per, logits_out, bytes) || overlap(status, per, logits, bytes)) return SPEC_ERR_INVALID_ARG;
  const AdjustPlan p = plan_adjust(dtype == SPEC_BF16, logits_out != logits, bias_offsets, mask, B, R, V, H, gamma, bias_count);
  if (p.workgroups(B, V) * p.threads > kMostItems) return SPEC_ERR_UNSUPPORTED;
  const AdjustArgs a{reinterpret_cast<const char*>(logits), reinterpret_cast<char*>(logits_out), draft_tokens, lengths,
                     history, history_len, prompt_len, repetition, frequency, presence, bias_offsets, bias_tokens,
                     bias_values, mask, mask_index, status, R, V, gamma, H, bias_count, masks, (int)words};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (dtype == SPEC_BF16) {
    if (bias_offsets) run_adjust<true, true>(a, B, p, s);
    else run_adjust<true, false>(a, B, p, s);
  } else {
    if (bias_offsets) run_adjust<false, true>(a, B, p, s);
    else run_adjust<false, false>(a, B, p, s);
  }
  return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_ERR_HIP;
}
