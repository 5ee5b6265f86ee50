// Penalties, biases and masks on logits, row by row of a draft block, on gfx950.
//
//   count of row k = the token's occurrences in the request's output and in the draft tokens before row k
//   z = z > 0 ? z / repetition : z * repetition   (a token of the prompt, or of count > 0)
//   z = z - frequency * count;  z = z - presence (count > 0);  z = z + bias;  z = -inf where the mask's bit is 0
//
// Nearly all of a row stays as it is: a history names a few thousand tokens of the vocabulary.  A workgroup takes a
// request and a slice of the vocabulary: it counts the slice's tokens of the history in LDS (a word per token; the
// first to name a token puts it on a list), and then goes over the list for every row of the block.  In place the
// rest of the row is touched only where a mask forbids it; out of place it is copied.  The rows of a block share
// one count, the draft tokens before a row are compared with the listed token one by one.
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

constexpr int kThreads = 256;
constexpr int kSlice = 8192;                 // tokens of the vocabulary per workgroup (at most 2^16)
constexpr uint32_t kInPrompt = 1u << 30, kListed = 1u << 31, kCount = kInPrompt - 1;

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

// The row's mask bits of tokens v .. v + 31 (0 past the words).
__device__ __forceinline__ uint32_t mask_bits(const uint32_t* m, int words, int v) {
  const int w = v >> 5, s = v & 31;
  const uint32_t lo = m[w], hi = w + 1 < words ? m[w + 1] : 0u;
  return (uint32_t)((((uint64_t)hi << 32) | lo) >> s);
}

template <bool BF16>
__device__ __forceinline__ void store_elem(char* row, int64_t v, float z) {
  if constexpr (BF16) reinterpret_cast<__bf16*>(row)[v] = (__bf16)z;
  else reinterpret_cast<float*>(row)[v] = z;
}

// BIAS: the slots of the biases lie behind the counts.
template <bool BF16, bool BIAS, bool COPY>
__global__ __launch_bounds__(kThreads) void adjust_kernel(AdjustArgs a) {
  constexpr int ES = BF16 ? 2 : 4, VE = 16 / ES;
  constexpr uint32_t kNegInf = BF16 ? 0xff80ff80u : 0xff800000u;
  __shared__ uint32_t count[kSlice];
  __shared__ uint32_t bias_at[BIAS ? kSlice : 1];   // entry of the list + 1 (the last one of a token named twice)
  __shared__ uint16_t list[kSlice];
  __shared__ int32_t drafts[SPEC_MAX_GAMMA];
  __shared__ int listed, bad;
  const int tid = threadIdx.x, V = a.V, R = a.R, slices = (V + kSlice - 1) / kSlice;
  const int b = (int)(blockIdx.x / (unsigned)slices), slice = (int)(blockIdx.x % (unsigned)slices);
  const int v0 = slice * kSlice, n = min(kSlice, V - v0);

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

  for (int i = tid; i < n; i += kThreads) {
    count[i] = 0;
    if constexpr (BIAS) bias_at[i] = 0;
  }
  if (tid == 0) listed = bad = 0;
  const int need = penal ? min(live - 1, a.gamma) : 0;   // draft tokens that precede a live row
  if (tid < need) drafts[tid] = a.draft_tokens[(size_t)b * a.gamma + tid];
  __syncthreads();
  bool off = false;
  auto note = [&](int i, uint32_t old) {
    if (old == 0) list[atomicAdd(&listed, 1)] = (uint16_t)i;
  };
  if (penal && live > 0) {
    const int32_t* h = a.history + (size_t)b * a.H;
    for (int i = tid; i < hl; i += kThreads) {
      const int t = h[i], at = t - v0;
      off |= t < -1 || t >= V;
      if (at >= 0 && at < n) note(at, i < pl ? atomicOr(&count[at], kInPrompt) : atomicAdd(&count[at], 1u));
    }
    if (tid < need) {
      const int t = drafts[tid], at = t - v0;
      off |= t < 0 || t >= V;
      if (at >= 0 && at < n) note(at, atomicOr(&count[at], kListed));
    }
  }
  if constexpr (BIAS) {
    for (int i = tid; i < bn && live > 0; i += kThreads) {
      const int t = a.bias_tokens[bo + i], at = t - v0;
      off |= t < 0 || t >= V;
      if (at >= 0 && at < n) {
        note(at, atomicOr(&count[at], kListed));
        atomicMax(&bias_at[at], (uint32_t)i + 1);
      }
    }
  }
  if (off) bad = 1;
  __syncthreads();
  if (bad) st |= SPEC_REQ_BAD_TOKEN;
  if (slice == 0 && tid == 0 && a.status) a.status[b] = st;
  if (st) return;

  const uint32_t* mask = mi >= 0 ? a.mask + (size_t)mi * R * a.words : nullptr;
  if (COPY || mask) {
    for (int r = 0; r < live; ++r) {
      const size_t row = ((size_t)b * R + r) * V;
      const char* src = a.logits + row * ES;
      char* dst = a.out + row * ES;
      const uint32_t* m = mask ? mask + (size_t)r * a.words : nullptr;
      // vectors that lie within the slice; up to VE - 1 values before and after them
      const int head = min((int)((0 - (row + v0)) & (VE - 1)), n), nv = (n - head) / VE, rest = n - head - nv * VE;
      for (int i = tid; i < nv; i += kThreads) {
        const int v = v0 + head + i * VE;
        const uint32_t on = m ? mask_bits(m, a.words, v) & ((1u << VE) - 1) : (1u << VE) - 1;
        if (!COPY && on == (1u << VE) - 1) continue;
        v4u32 z = {};
        if (on) z = __builtin_nontemporal_load(reinterpret_cast<const v4u32*>(src + (size_t)v * ES));
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          if constexpr (BF16) {
            const uint32_t p = on >> (2 * x) & 3u, keep = (p & 1u ? 0xffffu : 0u) | (p & 2u ? 0xffff0000u : 0u);
            z[x] = (z[x] & keep) | (kNegInf & ~keep);
          } else {
            z[x] = on >> x & 1u ? z[x] : kNegInf;
          }
        }
        *reinterpret_cast<v4u32*>(dst + (size_t)v * ES) = z;
      }
      if (tid < head + rest) {
        const int v = v0 + (tid < head ? tid : tid + nv * VE);
        const bool on = !m || (m[v >> 5] >> (v & 31) & 1u);
        if (!on) store_elem<BF16>(dst, v, -INFINITY);
        else if (COPY) store_elem<BF16>(dst, v, load_elem<BF16>(src, v));
      }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the copy is written before values of it are written again
    __syncthreads();
  }
  const unsigned E = (unsigned)listed, pairs = E * (unsigned)live;
  constexpr int U = 4;   // values in flight per thread
  for (unsigned p0 = tid; p0 < pairs; p0 += U * kThreads) {
    float z[U];
    size_t at[U];
    bool on[U];
    unsigned e[U];
    int r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const unsigned p = p0 + u * kThreads;
      on[u] = p < pairs;
      r[u] = on[u] ? (int)(p / E) : 0;
      e[u] = on[u] ? list[p - (unsigned)r[u] * E] : 0u;
      const int v = v0 + (int)e[u];
      if (mask && on[u]) on[u] = mask[(size_t)r[u] * a.words + (v >> 5)] >> (v & 31) & 1u;
      at[u] = ((size_t)b * R + r[u]) * V + v;
      z[u] = on[u] ? load_elem<BF16>(a.logits, (int64_t)at[u]) : 0.f;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!on[u]) continue;
      const uint32_t word = count[e[u]];
      int c = (int)(word & kCount);
      const int v = v0 + (int)e[u], before = min(r[u], need);
      for (int k = 0; k < before; ++k) c += drafts[k] == v;
      float x = z[u];
      if (c > 0 || (word & kInPrompt)) x = x > 0.f ? x / rep : x * rep;
      x = x - freq * (float)c;
      if (c > 0) x = x - pres;
      if constexpr (BIAS) {
        const uint32_t k = bias_at[e[u]];
        if (k) x = x + a.bias_values[bo + (int)k - 1];
      }
      store_elem<BF16>(a.out, (int64_t)at[u], x);
    }
  }
}

template <bool BF16, bool BIAS>
void run_adjust(const AdjustArgs& a, int B, hipStream_t s) {
  const dim3 grid((unsigned)ceil_div(a.V, kSlice) * (unsigned)B);
  if (a.logits == a.out) hipLaunchKernelGGL((adjust_kernel<BF16, BIAS, false>), grid, dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL((adjust_kernel<BF16, BIAS, true>), grid, dim3(kThreads), 0, s, a);
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
  // a launch's work-items are counted in 32 bits
  if ((long long)ceil_div(V, kSlice) * B * kThreads > 0xffffffffll) return SPEC_ERR_UNSUPPORTED;
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
