// What stands between a row of logits and the choice of its next token: penalties for
// repeated tokens, biases, and the mask of a grammar, in one pass.
//
//   z = logits[v];  c = how often v stands in the generated part of the history
//   v stands in the history at all:   z = z > 0 ? z / repetition : z * repetition
//   z = z - (frequency * c + presence * [c > 0]) + the sum of v's biases
//   v is not allowed:                 z = -inf
//
// A block takes some slices of a row's vocabulary, one after the other, and counts in shared memory
// what of the history lies in each. The counts are not cleared beforehand, which would take as many
// accesses as the logits themselves: a bit for each token says whether its count
// means anything, and only the counts of tokens that occur are set to zero first. The next slice's
// logits are loaded, and its counts taken, around this one's arithmetic. A history of up to 4096 tokens is
// first put into lists by slices, so that a slice's counts cost what lies in it; a longer one is read
// again for each slice. (256 rows of 131072 fp32 and a history of 2048: one slice a block, the history
// read for each, 88 us; several slices a block, each looking through the whole history, 92; as it is 82,
// 3.3 TB/s: the counts and their barriers leave memory waiting, without penalties it is 68 and without biases
// too 54.)
#pragma once

#include <stdint.h>

#include "lm_rows.cuh"

namespace gws {

constexpr int LOGIT_THREADS = 512;
constexpr int LOGIT_STEP = LOGIT_THREADS * GROUP;   // tokens that a block's threads take at once
constexpr int LOGIT_GROUPS = 2;                     // groups of a thread in a slice, at most
constexpr int LOGIT_SLICE = LOGIT_GROUPS * LOGIT_STEP;
constexpr int MAX_BIASES = 1024;                    // of a row
constexpr int TOKENS_AHEAD = 8;                     // tokens of the history that a thread loads at once
constexpr int LISTED = TOKENS_AHEAD * LOGIT_THREADS;
constexpr int MAX_LISTS = 64;                       // slices of a block, at most
constexpr uint32_t SEEN = 1u << 31;                 // a count's top bit: the token stands in the prompt

struct LogitParams {
  const void* logits;
  void* out;
  int64_t ldl, ldo;
  int64_t rows;
  int vocab;
  int slice, slices;                 // tokens of a slice, a multiple of LOGIT_STEP up to LOGIT_SLICE; slices of a row
  int shift;                         // slice is 1 << shift
  int each, blocks;                  // slices of a block, at most MAX_LISTS; blocks of a row
  int lists;                         // the history is put into lists first: more than one slice, up to LISTED tokens
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
__global__ void __launch_bounds__(LOGIT_THREADS, 2) adjust_logits_kernel(const __grid_constant__ LogitParams p) {
  extern __shared__ __align__(16) uint32_t logit_smem[];
  constexpr bool WHOLE = PATH != ANY;
  // Twice each: counts, the bits that say which of them mean something, and the tokens with biases; and the
  // row's biases.
  const int words = p.slice / 32;
  uint32_t* const counts = logit_smem;
  uint32_t* const knowns = counts + (p.tokens ? 2 * p.slice : 0);
  uint32_t* const biaseds = knowns + (p.tokens ? 2 * words : 0);
  int* const bias_at = reinterpret_cast<int*>(biaseds + (p.biases ? 2 * words : 0));
  float* const bias_value = reinterpret_cast<float*>(bias_at + p.biases);
  uint32_t* const list = reinterpret_cast<uint32_t*>(bias_value + p.biases);
  __shared__ int list_at[MAX_LISTS + 1], list_size[MAX_LISTS];
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
  // a token's place in the slice that begins at `base`, where it is below p.slice; no token is -1
  auto local = [](int token, int base) { return static_cast<uint32_t>(token) - static_cast<uint32_t>(base); };
  const uint32_t width = p.slice;
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
  // A round of the history: this thread's tokens, -1 for what does not count.
  int length = 0, prompt = 0;
  int token[TOKENS_AHEAD];
  auto load_tokens = [&](int base) {
    int64_t t[TOKENS_AHEAD];
#pragma unroll
    for (int j = 0; j < TOKENS_AHEAD; ++j) {
      const int i = base + j * LOGIT_THREADS + static_cast<int>(threadIdx.x);
      t[j] = i < length ? token_at(p.tokens, p.wide_tokens, row * p.ldt + i) : -1;
    }
#pragma unroll
    for (int j = 0; j < TOKENS_AHEAD; ++j) token[j] = t[j] >= 0 && t[j] < p.vocab ? static_cast<int>(t[j]) : -1;
  };
  load_logits(first);
  float rep = 1.0f, freq = 0.0f, pres = 0.0f;
  constexpr int ROUND = TOKENS_AHEAD * LOGIT_THREADS;
  int rounds = 0;
  if (p.tokens) {
    length = p.lengths ? min(max(p.lengths[row], 0), p.history) : p.history;
    prompt = p.prompts ? p.prompts[row] : 0;
    if (p.repetition) rep = p.repetition[row];
    if (p.frequency) freq = p.frequency[row];
    if (p.presence) pres = p.presence[row];
    rounds = (length + ROUND - 1) / ROUND;
    if (rounds == 1) load_tokens(0);
  }
  for (int i = threadIdx.x; i < p.biases; i += LOGIT_THREADS) {
    const int64_t t = token_at(p.bias_tokens, p.wide_biases, row * p.ldb + i);
    bias_at[i] = t >= 0 && t < p.vocab ? static_cast<int>(t) : -1;
    bias_value[i] = p.bias_values[row * p.ldv + i];
  }
  const bool counted = rounds > 0 || p.biases > 0;
  const bool lists = p.lists && rounds > 0;
  if (lists) {
    // Each token's place in its slice's list; the lists' begins; the lists.
    for (int i = threadIdx.x; i < MAX_LISTS; i += LOGIT_THREADS) list_size[i] = 0;
    __syncthreads();
    int rank[TOKENS_AHEAD];
    const uint32_t from = static_cast<uint32_t>(first) << p.shift, span = static_cast<uint32_t>(last - first) << p.shift;
#pragma unroll
    for (int j = 0; j < TOKENS_AHEAD; ++j) {
      const uint32_t at = static_cast<uint32_t>(token[j]) - from;
      rank[j] = token[j] >= 0 && at < span ? atomicAdd(list_size + (at >> p.shift), 1) : -1;
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      const int a = list_size[2 * threadIdx.x], b = list_size[2 * threadIdx.x + 1];
      int sum = a + b;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int left = __shfl_up_sync(0xffffffffu, sum, o);
        if (static_cast<int>(threadIdx.x) >= o) sum += left;
      }
      list_at[2 * threadIdx.x] = sum - a - b;
      list_at[2 * threadIdx.x + 1] = sum - b;
      if (threadIdx.x == 31) list_at[MAX_LISTS] = sum;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < TOKENS_AHEAD; ++j) {
      if (rank[j] < 0) continue;
      const uint32_t at = static_cast<uint32_t>(token[j]) - from;
      const bool of_prompt = j * LOGIT_THREADS + static_cast<int>(threadIdx.x) < prompt;
      list[list_at[at >> p.shift] + rank[j]] = (at & (width - 1)) | (of_prompt ? SEEN : 0);
    }
    __syncthreads();
  }
  // f(place, whether it is of the prompt) for the history's tokens in a slice.
  auto each_token = [&](int slice, auto f) {
    if (lists) {
      const int end = list_at[slice - first + 1];
      for (int i = list_at[slice - first] + threadIdx.x; i < end; i += LOGIT_THREADS)
        f(list[i] & ~SEEN, (list[i] & SEEN) != 0);
      return;
    }
    const int base = slice << p.shift;
    for (int r = 0; r < rounds; ++r) {
      if (rounds > 1) load_tokens(r * ROUND);
      const int left = length - r * ROUND;
#pragma unroll
      for (int j = 0; j < TOKENS_AHEAD; ++j) {
        if (j * LOGIT_THREADS >= left) break;
        const uint32_t at = local(token[j], base);
        if (at < width) f(at, r * ROUND + j * LOGIT_THREADS + static_cast<int>(threadIdx.x) < prompt);
      }
    }
  };
  // What a slice's counts need before they can be taken.
  auto clear = [&](int slice) {
    const int b = slice & 1;
    if (p.tokens)
      for (int i = threadIdx.x; i < words; i += LOGIT_THREADS) knowns[b * words + i] = 0;
    if (p.biases)
      for (int i = threadIdx.x; i < words; i += LOGIT_THREADS) biaseds[b * words + i] = 0;
    uint32_t* count = counts + b * p.slice;
    each_token(slice, [&](uint32_t at, bool) { count[at] = 0; });
  };
  auto take = [&](int slice) {
    const int b = slice & 1;
    uint32_t *count = counts + b * p.slice, *known = knowns + b * words, *biased = biaseds + b * words;
    each_token(slice, [&](uint32_t at, bool of_prompt) {
      if (of_prompt)
        atomicOr(count + at, SEEN);
      else
        atomicAdd(count + at, 1u);
      atomicOr(known + at / 32, 1u << (at % 32));
    });
    for (int i = threadIdx.x; i < p.biases; i += LOGIT_THREADS) {
      const uint32_t at = local(bias_at[i], slice * p.slice);
      if (at < width) atomicOr(biased + at / 32, 1u << (at % 32));
    }
  };
  if (counted) {
    clear(first);
    __syncthreads();
    take(first);
  }
  U* out = static_cast<U*>(p.out) + row * p.ldo;
  for (int slice = first; slice < last; ++slice) {
    Raw<T> now[LOGIT_GROUPS];
    uint32_t may[LOGIT_GROUPS];
#pragma unroll
    for (int k = 0; k < LOGIT_GROUPS; ++k) {
      now[k] = raw[k];
      may[k] = bits[k];
    }
    if (slice + 1 < last) load_logits(slice + 1);
    if (counted) {
      if (slice + 1 < last) clear(slice + 1);
      __syncthreads();
    }
    const int b = slice & 1;
    const uint32_t *count = counts + b * p.slice, *known = knowns + b * words, *biased = biaseds + b * words;
#pragma unroll
    for (int k = 0; k < LOGIT_GROUPS; ++k) {
      if (k * LOGIT_STEP >= p.slice) break;
      const int c = column(slice, k), c0 = c - slice * p.slice;
      const bool mine = c < p.vocab;
      uint32_t seen = 0, plus = 0;
      if (mine) {
        if (rounds > 0) seen = known[c0 / 32] >> (c0 % 32) & 0xFF;
        if (p.biases) plus = biased[c0 / 32] >> (c0 % 32) & 0xFF;
      }
      float z[GROUP];
      unpack(now[k], z);
      // One token after the other, in a loop that is rarely entered.
#pragma unroll 1
      for (uint32_t left = seen | plus; left; left &= left - 1) {
        const int i = __ffs(left) - 1;
        float v = 0.0f;
#pragma unroll
        for (int j = 0; j < GROUP; ++j) v = j == i ? z[j] : v;
        if (seen >> i & 1) {
          const uint32_t n = count[c0 + i];
          v = v > 0.0f ? v / rep : v * rep;
          if (n & ~SEEN) v -= fmaf(freq, static_cast<float>(n & ~SEEN), pres);
        }
        if (plus >> i & 1) {
          float add = 0.0f;
          for (int j = 0; j < p.biases; ++j)
            if (bias_at[j] == c + i) add += bias_value[j];
          v += add;
        }
#pragma unroll
        for (int j = 0; j < GROUP; ++j) z[j] = j == i ? v : z[j];
      }
      if (p.allowed) {
        const uint32_t mask = may[k] >> (c % 32);
#pragma unroll
        for (int i = 0; i < GROUP; ++i) z[i] = mask & 1u << i ? z[i] : -INFINITY;
      }
      if (PATH == ANY || mine)
        store_group<WHOLE>(out, c, p.vocab, threadIdx.x, LOGIT_THREADS, pack<U>(z));
    }
    if (counted && slice + 1 < last) {
      take(slice + 1);
      __syncthreads();   // this slice's counts have been read
    }
  }
}

}  // namespace gws
