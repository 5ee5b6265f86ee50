// Penalties, biases and masks on logits, row by row of a draft block, on gfx950.
//
//   count of row k = the token's occurrences in the request's output and in the draft tokens before row k
//   z = z > 0 ? z / repetition : z * repetition   (a token of the prompt, or of count > 0)
//   z = z - frequency * count;  z = z - presence (count > 0);  z = z + bias;  z = -inf where the mask's bit is 0
//
// Nearly all of a row stays as it is: a history names a few thousand tokens of the vocabulary.  A workgroup takes a
// request and a slice of the vocabulary.  It counts the slice's tokens of the history in LDS (a word per token; the
// first to count a token puts it on a list), and then goes through the block's rows, which share one count; the draft
// tokens before a row are compared with the listed token one by one.
//   Out of place, under a mask, or where much may be listed: the slice of a row goes through LDS, where
//   lanes take the listed tokens (adjusted in the registers that carry the rows, a lane here and there of every wave,
//   it took as long as the copy itself).  Masks are applied on the way out.  In place, pieces without a count are
//   written only where the mask forbids a value, and read only where it forbids some.
//   In place without a mask and with few tokens: lanes take pairs of listed token and row in memory.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <utility>

#include "common.hpp"
#include "rowseg.hpp"
#include "spec_verify.h"
#include "xent_plan.hpp"

namespace spec {
namespace {

constexpr int kSlice = 4096, kLongHistory = 8192;
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

// S tokens of the vocabulary and T threads per workgroup.
enum { kCopy = 0, kPlace = 1, kFew = 2 };   // out of place; in place; in place without a mask, few tokens

template <bool BF16, bool BIAS, int MODE, int S, int T, int U>
__global__ __launch_bounds__(T) void adjust_kernel(AdjustArgs a) {
  constexpr bool COPY = MODE == kCopy;
  constexpr int ES = BF16 ? 2 : 4, VE = 16 / ES, NV = S / VE / T;   // pieces of a row per lane; U rows at a time
  static_assert(S % (VE * T) == 0 && S <= 65536, "slice");
  __shared__ __attribute__((aligned(16))) uint32_t count[S];
  __shared__ __attribute__((aligned(16))) uint32_t bias_at[BIAS ? S : 4];   // entry of the list + 1 (the last one of a token named twice)
  __shared__ __attribute__((aligned(16))) char rows[MODE == kFew ? 1 : U][MODE == kFew ? 16 : S * ES];
  __shared__ uint16_t list[S];
  __shared__ int32_t drafts[SPEC_MAX_GAMMA];
  __shared__ int listed, bad;
  const int tid = threadIdx.x, V = a.V, R = a.R, slices = (V + S - 1) / S;
  const int b = (int)(blockIdx.x / (unsigned)slices), slice = (int)(blockIdx.x % (unsigned)slices);
  const int v0 = slice * S, n = min(S, V - v0);

  // the request's own numbers; every workgroup of the request comes to the same verdict
  int st = 0;
  const int L = a.lengths ? a.lengths[b] : a.gamma;
  if (L < 0 || L > a.gamma) st |= SPEC_REQ_BAD_LENGTH;
  const int live = st ? 0 : L + (R - a.gamma);
  int hl = a.history ? (a.history_len ? a.history_len[b] : a.H) : 0, pl = a.history && a.prompt_len ? a.prompt_len[b] : 0;
  if (hl < 0 || hl > a.H || pl < 0 || pl > hl) {
    st |= SPEC_REQ_BAD_LENGTH;
    hl = pl = 0;
  }
  const float rep = a.repetition ? a.repetition[b] : 1.f, freq = a.frequency ? a.frequency[b] : 0.f,
              pres = a.presence ? a.presence[b] : 0.f;
  if (!(rep > 0.f && rep < INFINITY && fabsf(freq) < INFINITY && fabsf(pres) < INFINITY)) st |= SPEC_REQ_BAD_PENALTY;
  const bool penal = rep != 1.f || freq != 0.f || pres != 0.f;   // else neither history nor drafts matter
  int bo = 0, bn = 0;
  if constexpr (BIAS) {
    bo = a.bias_offsets[b];
    const int be = a.bias_offsets[b + 1];
    if (bo < 0 || be < bo || be > a.bias_count) st |= SPEC_REQ_BAD_LIST;
    else bn = be - bo;
  }
  const int mi = a.mask ? (a.mask_index ? a.mask_index[b] : b) : -1;
  if (mi < -1 || mi >= a.masks) st |= SPEC_REQ_BAD_MASK;

  for (int i = tid; i < S / 4; i += T) {
    reinterpret_cast<v4u32*>(count)[i] = v4u32{};
    if constexpr (BIAS) reinterpret_cast<v4u32*>(bias_at)[i] = v4u32{};
  }
  if (tid == 0) listed = bad = 0;
  const int need = penal ? min(live - 1, a.gamma) : 0;   // draft tokens that precede a live row
  if (tid < need) drafts[tid] = a.draft_tokens[(size_t)b * a.gamma + tid];
  __syncthreads();
  bool off = false;
  auto note = [&](unsigned i, uint32_t old) {
    if (old == 0) list[atomicAdd(&listed, 1)] = (uint16_t)i;
  };
  if (penal && live > 0) {
    const int32_t* h = a.history + (size_t)b * a.H;
    // four tokens a load, F loads in flight per thread
    constexpr int F = 4;
    const int quads = hl >> 2;
    uint32_t most = 0;   // of t + 1: -1 is a hole
    auto count_in = [&](int t, int i) {
      const unsigned at = (unsigned)t - (unsigned)v0;
      most = max(most, (unsigned)t + 1u);
      if (at < (unsigned)n) note(at, i < pl ? atomicOr(&count[at], kInPrompt) : atomicAdd(&count[at], 1u));
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
    if (tid < (hl & 3)) count_in(h[4 * quads + tid], 4 * quads + tid);
    off |= most > (unsigned)V;
    if (tid < need) {
      const unsigned t = (unsigned)drafts[tid], at = t - (unsigned)v0;
      off |= t >= (unsigned)V;
      if (at < (unsigned)n) note(at, atomicOr(&count[at], kDrafted));
    }
  }
  if constexpr (BIAS) {
    for (int i = tid; i < bn && live > 0; i += T) {
      const unsigned t = (unsigned)a.bias_tokens[bo + i], at = t - (unsigned)v0;
      off |= t >= (unsigned)V;
      if (at < (unsigned)n) {
        note(at, atomicOr(&count[at], kBiased));
        atomicMax(&bias_at[at], (uint32_t)i + 1);
      }
    }
  }
  if (off) bad = 1;
  __syncthreads();
  if (bad) st |= SPEC_REQ_BAD_TOKEN;
  if (slice == 0 && tid == 0 && a.status) a.status[b] = st;
  if (st) return;

  const int E = listed;
  const uint32_t* mask = mi >= 0 ? a.mask + (size_t)mi * R * a.words : nullptr;
  const size_t row0 = (size_t)b * R * V + v0;
  // a listed token: what is the same for every row
  struct Token {
    int i, c;
    bool prompt, drafted, biased;
    float bias;
  };
  auto token = [&](int e) {
    Token t;
    t.i = list[e];
    const uint32_t w = count[t.i];
    t.c = (int)(w & kCount);
    t.prompt = w & kInPrompt;
    t.drafted = w & kDrafted;
    t.biased = BIAS && (w & kBiased);
    t.bias = 0.f;
    if constexpr (BIAS)
      if (t.biased) t.bias = a.bias_values[bo + (int)bias_at[t.i] - 1];
    return t;
  };
  auto adjusted = [&](float z, const Token& t, int r) {
    int c = t.c;
    if (t.drafted)
      for (int k = 0; k < min(r, need); ++k) c += drafts[k] == v0 + t.i;
    if (c > 0 || t.prompt) z = z > 0.f ? z / rep : z * rep;
    if (c > 0) {
      z = z - freq * (float)c;
      z = z - pres;
    }
    if (t.biased) z = z + t.bias;
    return z;
  };

  if constexpr (MODE == kFew) {
    const unsigned pairs = (unsigned)E * (unsigned)live;
    for (unsigned p0 = tid; p0 < pairs; p0 += U * T) {
      float z[U];
      Token t[U];
      int r[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const unsigned p = min(p0 + u * T, pairs - 1);
        r[u] = (int)(p / (unsigned)E);
        t[u] = token((int)(p % (unsigned)E));
        z[u] = load_elem<BF16>(a.logits, (int64_t)(row0 + (size_t)r[u] * V + t[u].i));
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (p0 + u * T < pairs) store_elem<BF16>(a.out, (int64_t)(row0 + (size_t)r[u] * V + t[u].i), adjusted(z[u], t[u], r[u]));
    }
  } else {

    constexpr uint32_t kAll = (1u << VE) - 1;
    uint32_t some[NV];   // in place: a lane's values with a count
#pragma unroll
    for (int q = 0; q < NV; ++q) {
      some[q] = 0;
      if (!COPY)
#pragma unroll
        for (int x = 0; x < VE; ++x) some[q] |= (count[(tid + q * T) * VE + x] ? 1u : 0u) << x;
    }
    Token mine{};   // the lane's first listed token
    if (tid < E) mine = token(tid);
    for (int r0 = 0; r0 < live; r0 += U) {
      v4u32 z[U][NV];
      uint32_t on[U][NV];   // allowed values of the piece (0 where there is none)
      bool move[U][NV];     // in place only what changes is read: a value with a count, or one beside a forbidden one
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int q = 0; q < NV; ++q) {
          const int i = (tid + q * T) * VE, left = r0 + u < live ? n - i : 0;
          on[u][q] = left >= VE ? kAll : left > 0 ? (1u << left) - 1 : 0u;
          if (mask && left > 0) on[u][q] &= mask[(size_t)(r0 + u) * a.words + ((v0 + i) >> 5)] >> ((v0 + i) & 31);
        }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int q = 0; q < NV; ++q) {
          const int i = (tid + q * T) * VE;
          const uint32_t whole = i + VE <= n ? kAll : (1u << max(n - i, 0)) - 1;
          move[u][q] = COPY ? on[u][q] != 0 : (on[u][q] & some[q]) != 0 || (on[u][q] != 0 && on[u][q] != whole);
          if (!move[u][q]) continue;
          const size_t at = row0 + (size_t)(r0 + u) * V + i;
          if (i + VE <= n) {
            z[u][q] = __builtin_nontemporal_load(&reinterpret_cast<const Piece<ES>*>(a.logits + at * ES)->v);
          } else {   // the row's last values
            z[u][q] = v4u32{};
            for (int x = 0; i + x < n; ++x) {
              const uint32_t h = BF16 ? reinterpret_cast<const uint16_t*>(a.logits)[at + x] : reinterpret_cast<const uint32_t*>(a.logits)[at + x];
              if constexpr (BF16) {
                if (x < 2) z[u][q].x |= h << (16 * x);
                else if (x < 4) z[u][q].y |= h << (16 * (x - 2));
                else if (x < 6) z[u][q].z |= h << (16 * (x - 4));
                else z[u][q].w |= h << (16 * (x - 6));
              } else {
                if (x == 0) z[u][q].x = h;
                else if (x == 1) z[u][q].y = h;
                else z[u][q].z = h;
              }
            }
          }
        }
      if (E > 0) {
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int q = 0; q < NV; ++q)
            if (move[u][q]) *reinterpret_cast<v4u32*>(&rows[u][(tid + q * T) * 16]) = z[u][q];
        __syncthreads();
        for (int e = tid; e < E; e += T) {
          const Token t = e == tid ? mine : token(e);
#pragma unroll
          for (int u = 0; u < U; ++u)
            if (r0 + u < live) store_elem<BF16>(rows[u], t.i, adjusted(load_elem<BF16>(rows[u], t.i), t, r0 + u));
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int q = 0; q < NV; ++q)
            if (move[u][q]) z[u][q] = *reinterpret_cast<const v4u32*>(&rows[u][(tid + q * T) * 16]);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int q = 0; q < NV; ++q) {
          const int i = (tid + q * T) * VE;
          if (r0 + u >= live || i >= n || (!COPY && !move[u][q] && on[u][q] != 0)) continue;
          const size_t at = row0 + (size_t)(r0 + u) * V + i;
          v4u32 y = move[u][q] ? z[u][q] : v4u32{};
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            if constexpr (BF16) {
              const uint32_t p = on[u][q] >> (2 * x) & 3u, keep = (p & 1u ? 0xffffu : 0u) | (p & 2u ? 0xffff0000u : 0u);
              y[x] = (y[x] & keep) | (0xff80ff80u & ~keep);
            } else {
              y[x] = on[u][q] >> x & 1u ? y[x] : 0xff800000u;
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
}

template <bool BF16, bool BIAS, int MODE, int S, int T, int U>
void launch(const AdjustArgs& a, int B, hipStream_t s) {
  const dim3 grid((unsigned)ceil_div(a.V, S) * (unsigned)B);
  hipLaunchKernelGGL((adjust_kernel<BF16, BIAS, MODE, S, T, U>), grid, dim3(T), 0, s, a);
}

// Slices of 4096 tokens by 512 threads, one row of it in LDS at a time: 24 waves a CU or more (64 blocks of 17 rows of
// 151936 bf16, half of them live, out of place: 90 us; two rows at a time 98; slices of 2048 by 256 threads 96, of
// 8192 by 1024 118).  Every slice's workgroup reads the whole history, and from some 8000 tokens on half as many
// slices are faster, where their LDS leaves two workgroups to a CU (96 x 8 rows of 129280 after 30011 tokens:
// 120 -> 108 us; after 1000: 74 -> 77).
// In place, listed tokens cost 30 ps a row where they lie in memory, and a row's slice through LDS 1 ps a token: where
// the history can name a thirtieth of the vocabulary the row goes through LDS.
template <bool BF16, bool BIAS>
void run_adjust(const AdjustArgs& a, int B, hipStream_t s) {
  const bool copy = a.logits != a.out;
  if (!copy && !a.mask && a.H <= a.V / 32) {
    launch<BF16, BIAS, kFew, kSlice, 512, 4>(a, B, s);
    return;
  }
  if constexpr (BF16 && !BIAS) {
    if (a.H > kLongHistory) {
      if (copy) launch<BF16, BIAS, kCopy, 2 * kSlice, 1024, 1>(a, B, s);
      else launch<BF16, BIAS, kPlace, 2 * kSlice, 1024, 1>(a, B, s);
      return;
    }
  }
  if (copy) launch<BF16, BIAS, kCopy, kSlice, 512, 1>(a, B, s);
  else launch<BF16, BIAS, kPlace, kSlice, 512, 1>(a, B, s);
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
  // a launch's work-items are counted in 32 bits; the larger slices have the more of them
  if ((long long)ceil_div(V, 2 * kSlice) * B * 1024 > 0xffffffffll) return SPEC_ERR_UNSUPPORTED;
  const AdjustArgs a{reinterpret_cast<const char*>(logits), reinterpret_cast<char*>(logits_out), draft_tokens, lengths,
                     history, history_len, prompt_len, repetition, frequency, presence, bias_offsets, bias_tokens,
                     bias_values, mask, mask_index, status, R, V, gamma, H, bias_count, masks, (int)words};
  hipStream_t s = reinterpret_cast<hipStream_t>(stream);
  if (dtype == SPEC_BF16) {
    if (bias_offsets) run_adjust<true, true>(a, B, s);
    else run_adjust<true, false>(a, B, s);
  } else {
    if (bias_offsets) run_adjust<false, true>(a, B, s);
    else run_adjust<false, false>(a, B, s);
  }
  return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_ERR_HIP;
}
