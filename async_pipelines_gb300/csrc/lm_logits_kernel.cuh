// What stands between a row of logits and the choice of its next token: penalties for
// repeated tokens, biases, and the mask of a grammar, in one pass.
//
//   z = logits[v];  c = how often v stands in the generated part of the history
//   v stands in the history at all:   z = z > 0 ? z / repetition : z * repetition
//   z = z - (frequency * c + presence * [c > 0]) + the sum of v's biases
//   v is not allowed:                 z = -inf
//
// A block takes a slice of a row's vocabulary and counts in shared memory what of the
// history lies in it. The counts are not cleared beforehand, which would take as many
// accesses as the logits themselves: a bit for each token says whether its count
// means anything, and only the counts of tokens that occur are set to zero first.
#pragma once

#include <stdint.h>

#include "lm_rows.cuh"

namespace gws {

constexpr int LOGIT_THREADS = 256;
constexpr int LOGIT_STEP = LOGIT_THREADS * GROUP;   // tokens that a block's threads take at once
constexpr int MAX_BIASES = 1024;                    // of a row
constexpr uint32_t SEEN = 1u << 31;                 // a count's top bit: the token stands in the prompt

struct LogitParams {
  const void* logits;
  void* out;
  int64_t ldl, ldo;
  int64_t rows;
  int vocab;
  int slice, slices;                 // tokens of a block, a multiple of LOGIT_STEP; blocks of a row
  const void* tokens;                // rows x history, or NULL
  int64_t ldt;
  int wide_tokens;                   // int64, else int32
  int history;
  const int *lengths, *prompts;      // NULL: history; 0
  const float *repetition, *frequency, *presence;   // NULL: 1, 0, 0
  const void* bias_tokens;           // rows x biases, or NULL
  const float* bias_values;
  int64_t ldb, ldv;
  int wide_biases;
  int biases;
  const uint32_t* allowed;           // rows x ceil(vocab / 32), or NULL
  int64_t lda;
};

__device__ __forceinline__ int64_t token_at(const void* p, int wide, int64_t i) {
  return wide ? static_cast<const int64_t*>(p)[i] : static_cast<const int*>(p)[i];
}

// T: the logits' type; U: the output's.
template <typename T, typename U, Path PATH>
__global__ void __launch_bounds__(LOGIT_THREADS) adjust_logits_kernel(const __grid_constant__ LogitParams p) {
  extern __shared__ __align__(16) uint32_t logit_smem[];
  __shared__ int chunk_count[LOGIT_THREADS / 32];
  constexpr bool WHOLE = PATH != ANY;
  // counts, the bits that say which of them mean something, the tokens with biases, and those
  uint32_t* count = logit_smem;
  uint32_t* known = count + (p.tokens ? p.slice : 0);
  uint32_t* biased = known + (p.tokens ? p.slice / 32 : 0);
  int* bias_at = reinterpret_cast<int*>(biased + (p.biases ? p.slice / 32 : 0));
  float* bias_value = reinterpret_cast<float*>(bias_at + p.biases);
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t row = blockIdx.x / p.slices;
  const int first = static_cast<int>(blockIdx.x % p.slices) * p.slice;
  const int width = min(p.slice, p.vocab - first);   // tokens of this slice
  auto local = [&](int64_t v) {   // a token's place in the slice, or -1
    const int64_t at = v - first;
    return at >= 0 && at < width ? static_cast<int>(at) : -1;
  };
  for (int i = threadIdx.x; i < p.slice / 32; i += LOGIT_THREADS) {
    if (p.tokens) known[i] = 0;
    if (p.biases) biased[i] = 0;
  }
  int length = 0, prompt = 0;
  float rep = 1.0f, freq = 0.0f, pres = 0.0f;
  if (p.tokens) {
    length = p.lengths ? min(max(p.lengths[row], 0), p.history) : p.history;
    prompt = p.prompts ? p.prompts[row] : 0;
    if (p.repetition) rep = p.repetition[row];
    if (p.frequency) freq = p.frequency[row];
    if (p.presence) pres = p.presence[row];
    for (int i = threadIdx.x; i < length; i += LOGIT_THREADS) {
      const int at = local(token_at(p.tokens, p.wide_tokens, row * p.ldt + i));
      if (at >= 0) count[at] = 0;
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < length; i += LOGIT_THREADS) {
    const int at = local(token_at(p.tokens, p.wide_tokens, row * p.ldt + i));
    if (at < 0) continue;
    if (i < prompt)
      atomicOr(count + at, SEEN);
    else
      atomicAdd(count + at, 1u);
    atomicOr(known + at / 32, 1u << (at % 32));
  }
  // the slice's biases, in the order in which they are given
  int biases = 0;
  for (int i0 = 0; i0 < p.biases; i0 += LOGIT_THREADS) {
    const int i = i0 + threadIdx.x;
    const int at = i < p.biases ? local(token_at(p.bias_tokens, p.wide_biases, row * p.ldb + i)) : -1;
    const unsigned vote = __ballot_sync(0xffffffffu, at >= 0);
    if ((threadIdx.x & 31) == 0) chunk_count[threadIdx.x / 32] = __popc(vote);
    __syncthreads();
    int to = biases + __popc(vote & ((1u << (threadIdx.x & 31)) - 1u));
    for (int w = 0; w < LOGIT_THREADS / 32; ++w) {
      if (w < static_cast<int>(threadIdx.x / 32)) to += chunk_count[w];
      biases += chunk_count[w];
    }
    if (at >= 0) {
      bias_at[to] = at;
      bias_value[to] = p.bias_values[row * p.ldv + i];
      atomicOr(biased + at / 32, 1u << (at % 32));
    }
    __syncthreads();
  }
  __syncthreads();
  const Row<T> in = row_of<T>(p.logits, row, p.rows, p.ldl);
  U* out = static_cast<U*>(p.out) + row * p.ldo;
  const uint32_t* allowed = p.allowed ? p.allowed + row * p.lda : nullptr;
  for (int c0 = threadIdx.x * GROUP; c0 - static_cast<int>(threadIdx.x) * GROUP < width; c0 += LOGIT_STEP) {
    const int c = c0 < width ? first + c0 : p.vocab;   // the row's end for a thread without a group
    const bool mine = c < p.vocab;
    Raw<T> raw = {};
    uint32_t bits = 0xFF, seen = 0, plus = 0;
    if (mine) {
      raw = load_group<WHOLE>(in, c, p.vocab);
      if (allowed) bits = allowed[c / 32] >> (c % 32) & 0xFF;
      if (p.tokens) seen = known[c0 / 32] >> (c0 % 32) & 0xFF;
      if (p.biases) plus = biased[c0 / 32] >> (c0 % 32) & 0xFF;
    }
    float z[GROUP];
    unpack(raw, z);
#pragma unroll
    for (int i = 0; i < GROUP; ++i) {
      if (seen >> i & 1) {
        const uint32_t n = count[c0 + i];
        z[i] = z[i] > 0.0f ? z[i] / rep : z[i] * rep;
        if (n & ~SEEN) z[i] -= fmaf(freq, static_cast<float>(n & ~SEEN), pres);
      }
      if (plus >> i & 1) {
        float add = 0.0f;
        for (int k = 0; k < biases; ++k)
          if (bias_at[k] == c0 + i) add += bias_value[k];
        z[i] += add;
      }
      if (!(bits >> i & 1)) z[i] = -INFINITY;
    }
    if (PATH == ANY || mine)
      store_group<WHOLE>(out, c, p.vocab, threadIdx.x, LOGIT_THREADS, pack<U>(z));
  }
}

}  // namespace gws
