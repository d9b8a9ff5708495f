// Host side of the logits' adjustments (include/gemm_ws_lm.h): argument checks, the slices
// of the vocabulary, and the launch.
#include <cstring>

#include "lm_host.cuh"
#include "lm_logits_kernel.cuh"

static_assert((gws::LOGIT_STEP & (gws::LOGIT_STEP - 1)) == 0 && (gws::LOGIT_GROUPS & (gws::LOGIT_GROUPS - 1)) == 0,
              "slices are powers of two, and so slots");

namespace {

constexpr size_t kSmemMost = 8 * (gws::MAX_SLOTS + gws::MAX_BIASES);

template <typename T, typename U>
int launch_logits(gemm_ws* h, bool fast, size_t smem, const gws::LogitParams& p, cudaStream_t s) {
  return launch_sized(
      h, fast ? gws::adjust_logits_kernel<T, U, gws::FAST> : gws::adjust_logits_kernel<T, U, gws::ANY>,
      p.rows * p.blocks, gws::LOGIT_THREADS, smem, kSmemMost, s, p);
}

}  // namespace

extern "C" {

int gemm_ws_adjust_logits(gemm_ws_t* h, int dtype, const void* logits, int64_t ldl, int out_dtype,
                          void* out, int64_t ldo, const void* tokens, int token_bytes, int64_t ldt,
                          int64_t history, const int32_t* lengths, const int32_t* prompt_lengths,
                          const float* repetition, const float* frequency, const float* presence,
                          const void* bias_tokens, int bias_token_bytes, int64_t ldb,
                          const float* bias_values, int64_t ldv, int64_t biases,
                          const uint32_t* allowed, int64_t lda, int64_t rows, int64_t vocab,
                          void* stream) {
  if (!h || dtype < GEMM_WS_BF16 || dtype > GEMM_WS_F32 ||
      (out_dtype != dtype && out_dtype != GEMM_WS_F32) || rows < 0 || rows > kMaxDim || vocab < 1 ||
      vocab > kMaxDim - 4096 || history < 0 || history > kMaxDim - 8192 || biases < 0 || biases > gws::MAX_BIASES)
    return GEMM_WS_ERR_INVALID_ARG;
  if (rows == 0) return GEMM_WS_OK;
  if (history == 0) tokens = nullptr;
  if (biases == 0) bias_tokens = nullptr;
  const int64_t words = ceil_div(vocab, 32);
  const Mat ml{logits, ldl, element_size(dtype)}, mo{out, ldo, element_size(out_dtype)},
      mt{tokens, ldt, token_bytes}, mb{bias_tokens, ldb, bias_token_bytes},
      mv{bias_tokens ? bias_values : nullptr, ldv, 4}, ma{allowed, lda, 4};
  if (!logits || !out || (history > 0 && !tokens) || (biases > 0 && (!bias_tokens || !bias_values)) ||
      (tokens && token_bytes != 4 && token_bytes != 8) ||
      (bias_tokens && bias_token_bytes != 4 && bias_token_bytes != 8))
    return GEMM_WS_ERR_INVALID_ARG;
  if (bad_matrix(ml, vocab) || bad_matrix(mo, vocab) || bad_matrix(mt, history) ||
      bad_matrix(mb, biases) || bad_matrix(mv, biases) || bad_matrix(ma, words))
    return GEMM_WS_ERR_INVALID_ARG;
  const void* vec[] = {lengths, prompt_lengths, repetition, frequency, presence};
  for (const void* v : vec)
    if (reinterpret_cast<uintptr_t>(v) % 4 != 0) return GEMM_WS_ERR_INVALID_ARG;
  // out may be the logits
  if (clash(mo, ml, rows, vocab, true)) return GEMM_WS_ERR_INVALID_ARG;
  const Span outputs[] = {span(mo, rows, vocab)};
  const Span inputs[] = {span(mt, rows, history), span(mb, rows, biases), span(mv, rows, biases),
                         span(ma, rows, words), {vec[0], rows * 4}, {vec[1], rows * 4}, {vec[2], rows * 4},
                         {vec[3], rows * 4}, {vec[4], rows * 4}};
  if (any_overlap(outputs, inputs)) return GEMM_WS_ERR_INVALID_ARG;
  gws::LogitParams q;
  std::memset(&q, 0, sizeof q);
  q.logits = logits;
  q.out = out;
  q.ldl = ldl;
  q.ldo = ldo;
  q.rows = rows;
  q.vocab = static_cast<int>(vocab);
  q.tokens = tokens;
  q.ldt = ldt;
  q.wide_tokens = token_bytes == 8;
  q.history = static_cast<int>(history);
  q.lengths = lengths;
  q.prompts = prompt_lengths;
  q.repetition = repetition;
  q.frequency = frequency;
  q.presence = presence;
  q.bias_tokens = bias_tokens;
  q.bias_values = bias_values;
  q.ldb = ldb;
  q.ldv = ldv;
  q.wide_biases = bias_token_bytes == 8;
  q.biases = bias_tokens ? static_cast<int>(biases) : 0;
  q.allowed = allowed;
  q.lda = lda;
  // Slices as long as they may be, but short enough that few rows still reach all SMs. Then as many of
  // them a block as cost least: memory is shared, so the time is that of all blocks' slices and begins by the
  // blocks held at once, but not less than one block's. What a block does for a history takes as long as
  // three slices, for biases alone half of one (256 rows of 131072 fp32 with 2048 tokens of history: 8 slices a
  // block 60 us, 16 70, 4 62; with biases alone 47, 63 and 48; 32 rows bf16: 4 slices 5.0, 8 6.6).
  // With a history too long for a hash table it is one slice.
  const int64_t steps = ceil_div(vocab, gws::LOGIT_STEP), held = gws::LOGIT_HELD * h->num_sms;
  int64_t per = gws::LOGIT_GROUPS;
  const int64_t spread = ceil_div(steps * rows, held);
  while (per > 1 && per > spread) per /= 2;
  q.slice = static_cast<int>(per * gws::LOGIT_STEP);
  q.slices = static_cast<int>(ceil_div(vocab, q.slice));
  q.blocks = q.slices;
  q.each = 1;
  const int64_t begin = tokens ? 12 : bias_tokens ? 2 : 1;   // quarters of a slice
  int64_t least = 0;
  if (history <= gws::LISTED)
    for (int64_t blocks = 1; blocks < 2 * q.slices; blocks *= 2) {
      const int64_t each = ceil_div(q.slices, blocks), there = ceil_div(q.slices, each);
      const int64_t cost = (rows * there > held ? rows * there : held) * (4 * each + begin);
      if (least != 0 && cost >= least) continue;
      least = cost;
      q.each = static_cast<int>(each);
      q.blocks = static_cast<int>(there);
    }
  if (rows * q.blocks > kMaxDim) return GEMM_WS_ERR_INVALID_ARG;
  q.slots = 64;
  while (q.slots < gws::MAX_SLOTS && q.slots < 2 * (history + q.biases)) q.slots *= 2;
  q.hashed = q.each > 1 || q.slots < q.slice;
  if (!q.hashed) q.slots = q.slice;
  const size_t smem = 8 * (tokens || q.biases ? q.slots + q.biases : 0);
  const bool fast = ml.wide() && mo.wide() && vocab % gws::GROUP == 0;
  DeviceGuard guard(h->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const bool same = out_dtype == dtype;
  switch (dtype) {
    case GEMM_WS_BF16:
      return same ? launch_logits<__nv_bfloat16, __nv_bfloat16>(h, fast, smem, q, s)
                  : launch_logits<__nv_bfloat16, float>(h, fast, smem, q, s);
    case GEMM_WS_F16:
      return same ? launch_logits<__half, __half>(h, fast, smem, q, s)
                  : launch_logits<__half, float>(h, fast, smem, q, s);
    default: return launch_logits<float, float>(h, fast, smem, q, s);
  }
}

}  // extern "C"
