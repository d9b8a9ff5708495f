// What stands between a row of logits and the choice of its next token: penalties for
// repeated tokens, biases, and the mask of a grammar, in one pass.
//
//   z = logits[v];  c = how often v stands in the generated part of the history
//   v stands in the history at all:   z = z > 0 ? z / repetition : z * repetition
//   z = z - (frequency * c + presence * [c > 0]) + the sum of v's biases
//   v is not allowed:                 z = -inf
//
// A block takes some slices of a row's vocabulary. What of the history and the biases lies in them it counts
// in a table in shared memory; the logits stream past that with nothing but the mask applied,
// and without a barrier; then the table's few tokens are computed from the logits once more and
// put over what the stream wrote. A history of up to 4096 tokens has a hash table of at least twice its tokens, so
// that a block may take many slices for one look at the history; a longer one is
// counted at its tokens' places in one slice. 256 rows of 131072 fp32 with a history of 2048: 60 us, 4.6 TB/s
// (biases alone 47, 5.8); the counting is latency that other blocks' streams cover in part. With counts looked up at
// each group of the stream, and so a barrier a slice, it was 82. Blocks of 256 threads, four an SM: 69.
#pragma once

#include <stdint.h>

#include "lm_rows.cuh"

namespace gws {

constexpr int LOGIT_THREADS = 512, LOGIT_HELD = 2;   // of a block; blocks of an SM
constexpr int LOGIT_STEP = LOGIT_THREADS * GROUP;   // tokens that a block's threads take at once
constexpr int LOGIT_GROUPS = 2;                     // groups of a thread in a slice, at most
constexpr int LOGIT_SLICE = LOGIT_GROUPS * LOGIT_STEP;
constexpr int MAX_BIASES = 1024;                    // of a row
constexpr int TOKENS_AHEAD = 8;                     // tokens of the history that a thread loads at once
constexpr int ROUND = TOKENS_AHEAD * LOGIT_THREADS; // of the block
constexpr int LISTED = 4096;                        // tokens of a history with a hash table
constexpr int MAX_SLOTS = 8192;                     // of a table
static_assert(LISTED + MAX_BIASES < MAX_SLOTS, "a search for a token meets an empty slot");
constexpr uint32_t TOP = 1u << 31;                  // of a count: the token stands in the prompt; of a key: it has biases
constexpr uint32_t EMPTY = TOP - 1;                 // no token: vocabularies are smaller

struct LogitParams {
  const void* logits;
  void* out;
  int64_t ldl, ldo;
  int64_t rows;
  int vocab;
  int slice, slices;                 // tokens of a slice, a multiple of LOGIT_STEP up to LOGIT_SLICE; slices of a row
  int each, blocks;                  // slices of a block; blocks of a row
  int slots;                         // of the table, a power of two
  int hashed;                        // tokens anywhere in the table; else each at its place in the block's one slice
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
__global__ void __launch_bounds__(LOGIT_THREADS, LOGIT_HELD) adjust_logits_kernel(const __grid_constant__ LogitParams p) {
  extern __shared__ __align__(16) uint32_t logit_smem[];
  constexpr bool WHOLE = PATH != ANY;
  uint32_t *const keys = logit_smem, *const counts = keys + p.slots;
  uint2* const biases = reinterpret_cast<uint2*>(counts + p.slots);   // token and value
  grid_dependency_wait();
  grid_launch_dependents();
  const int64_t row = blockIdx.x / p.blocks;
  const int first = static_cast<int>(blockIdx.x % p.blocks) * p.each, last = min(first + p.each, p.slices);
  const Row<T> in = row_of<T>(p.logits, row, p.rows, p.ldl);
  // the column of the thread's group k of a slice; the row's end where it has none
  auto column = [&](int slice, int k) {
    const int at = k * LOGIT_STEP + static_cast<int>(threadIdx.x) * GROUP;
    return at < p.slice && at < p.vocab - slice * p.slice ? slice * p.slice + at : p.vocab;
  };
  Raw<T> raw[LOGIT_GROUPS] = {};
  uint32_t bits[LOGIT_GROUPS];
  auto load_logits = [&](int slice) {
#pragma unroll
    for (int k = 0; k < LOGIT_GROUPS; ++k) {
      const int c = column(slice, k);
      bits[k] = ~0u;
      if (c < p.vocab) {
        raw[k] = load_group<WHOLE>(in, c, p.vocab);
        if (p.allowed) bits[k] = p.allowed[row * p.lda + c / 32];   // not looked at before it is needed
      }
    }
  };
  int length = 0;
  if (p.tokens) length = p.lengths ? min(max(p.lengths[row], 0), p.history) : p.history;
  const bool counted = length > 0 || p.biases > 0;
  // A round of the history, and of the biases, is on its way while the table is cleared.
  int64_t t[TOKENS_AHEAD];
  auto load_tokens = [&](int r) {
#pragma unroll
    for (int j = 0; j < TOKENS_AHEAD; ++j) {
      const int i = r + j * LOGIT_THREADS + static_cast<int>(threadIdx.x);
      t[j] = i < length ? token_at(p.tokens, p.wide_tokens, row * p.ldt + i) : -1;
    }
  };
  int64_t bias = -1;
  float value = 0.0f;
  auto load_bias = [&](int i) {
    if (i < p.biases) {
      bias = token_at(p.bias_tokens, p.wide_biases, row * p.ldb + i);
      value = p.bias_values[row * p.ldv + i];
    }
  };
  int prompt = 0;
  float rep = 1.0f, freq = 0.0f, pres = 0.0f;
  if (p.tokens) {
    if (p.prompts) prompt = p.prompts[row];
    if (p.repetition) rep = p.repetition[row];
    if (p.frequency) freq = p.frequency[row];
    if (p.presence) pres = p.presence[row];
  }
  const uint32_t base = static_cast<uint32_t>(first) * static_cast<uint32_t>(p.slice);
  if (counted) {
    load_tokens(0);
    load_bias(threadIdx.x);
    const uint32_t none = p.hashed ? EMPTY : 0;
    for (int i = threadIdx.x; i < p.slots; i += LOGIT_THREADS) {
      keys[i] = none;
      counts[i] = 0;
    }
    // The block's tokens are `span` from `base` on.
    const uint32_t width = static_cast<uint32_t>(p.slice) * static_cast<uint32_t>(last - first);
    const uint32_t span = min(width, static_cast<uint32_t>(p.vocab) - base);
    // A token's slot. Every block has more slots than tokens to put there.
    auto slot_of = [&](uint32_t token) {
      if (!p.hashed) return token - base;
      const uint32_t mask = p.slots - 1;
      uint32_t at = (token * 2654435761u >> 16) & mask;   // Knuth's multiplicative hash
      for (uint32_t i = 0; i < mask; ++i, at = (at + 1) & mask) {
        const uint32_t was = atomicCAS(keys + at, EMPTY, token);
        if (was == EMPTY || (was & ~TOP) == token) break;
      }
      return at;
    };
    __syncthreads();
    for (int r = 0; r < length; r += ROUND) {
      if (r > 0) load_tokens(r);
#pragma unroll
      for (int j = 0; j < TOKENS_AHEAD; ++j) {
        if (t[j] < base || t[j] - base >= span) continue;
        uint32_t* count = counts + slot_of(static_cast<uint32_t>(t[j]));
        if (r + j * LOGIT_THREADS + static_cast<int>(threadIdx.x) < prompt)
          atomicOr(count, TOP);
        else
          atomicAdd(count, 1u);
      }
    }
    for (int i = threadIdx.x; i < p.biases; i += LOGIT_THREADS) {
      if (i >= LOGIT_THREADS) load_bias(i);
      const bool mine = bias >= base && bias - base < span;
      biases[i] = make_uint2(mine ? static_cast<uint32_t>(bias) : ~0u, __float_as_uint(value));
      if (mine) atomicOr(keys + slot_of(static_cast<uint32_t>(bias)), TOP);
    }
  }
  U* out = static_cast<U*>(p.out) + row * p.ldo;
  load_logits(first);
  for (int slice = first; slice < last; ++slice) {
    Raw<T> now[LOGIT_GROUPS];
    uint32_t may[LOGIT_GROUPS];
#pragma unroll
    for (int k = 0; k < LOGIT_GROUPS; ++k) {
      now[k] = raw[k];
      may[k] = bits[k];
    }
    if (slice + 1 < last) load_logits(slice + 1);
#pragma unroll
    for (int k = 0; k < LOGIT_GROUPS; ++k) {
      if (k * LOGIT_STEP >= p.slice) break;
      const int c = column(slice, k);
      float z[GROUP];
      unpack(now[k], z);
      const uint32_t mask = may[k] >> (c % 32);
#pragma unroll
      for (int i = 0; i < GROUP; ++i) z[i] = mask & 1u << i ? z[i] : -INFINITY;
      if (PATH == ANY || c < p.vocab)
        store_group<WHOLE>(out, c, p.vocab, threadIdx.x, LOGIT_THREADS, pack<U>(z));
    }
  }
  if (!counted) return;
  __syncthreads();   // the table is complete, and what follows is written over what the stream wrote
  constexpr int AT_ONCE = 4;
  for (int i0 = threadIdx.x; i0 < p.slots; i0 += AT_ONCE * LOGIT_THREADS) {
    uint32_t n[AT_ONCE], may[AT_ONCE];
    int c[AT_ONCE];
    bool biased[AT_ONCE];
    T z[AT_ONCE];
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) {
      const int i = i0 + j * LOGIT_THREADS;
      n[j] = may[j] = 0;
      if (i >= p.slots) continue;
      const uint32_t key = keys[i];
      n[j] = counts[i];
      biased[j] = key & TOP;
      if (n[j] == 0 && !biased[j]) continue;
      c[j] = static_cast<int>(p.hashed ? key & ~TOP : base + i);
      may[j] = p.allowed ? p.allowed[row * p.lda + c[j] / 32] >> (c[j] % 32) & 1 : 1;
      z[j] = in.at[c[j]];   // where out is the logits, the stream has left what is allowed as it was
    }
#pragma unroll
    for (int j = 0; j < AT_ONCE; ++j) {
      if (!may[j]) continue;
      float v = to_float(z[j]);
      if (n[j] != 0) v = v > 0.0f ? v / rep : v * rep;
      if (n[j] & ~TOP) v -= fmaf(freq, static_cast<float>(n[j] & ~TOP), pres);
      if (biased[j]) {
        float add = 0.0f;
#pragma unroll 8
        for (int k = 0; k < p.biases; ++k) {
          const uint2 b = biases[k];
          add += b.x == static_cast<uint32_t>(c[j]) ? __uint_as_float(b.y) : 0.0f;
        }
        v += add;
      }
      out[c[j]] = round_to(v, U());
    }
  }
}

}  // namespace gws
