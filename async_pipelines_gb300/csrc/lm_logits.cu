// Host side of the logits' adjustments (include/gemm_ws_lm.h): argument checks, the slices
// of the vocabulary, and the launch.
#include <cstring>

#include "lm_host.cuh"
#include "lm_logits_kernel.cuh"

static_assert((gws::LOGIT_STEP & (gws::LOGIT_STEP - 1)) == 0 && (gws::LOGIT_GROUPS & (gws::LOGIT_GROUPS - 1)) == 0,
              "slices are powers of two");

namespace {

constexpr size_t kSmemMost = 4 * (2 * gws::LOGIT_SLICE + 4 * gws::LOGIT_SLICE / 32 + 2 * gws::MAX_BIASES +
                                   gws::LISTED);

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
  // them a block as leave the least work to the slowest SM, which holds two blocks: a block begins with
  // loads that wait for each other, which takes as long as about three slices, and where the
  // history does not fit the lists that is so for each slice.
  const int64_t steps = ceil_div(vocab, gws::LOGIT_STEP), held = 2 * h->num_sms;
  int64_t per = gws::LOGIT_GROUPS;
  const int64_t spread = ceil_div(steps * rows, held);
  if (per > spread) per = spread;
  q.slice = static_cast<int>(per * gws::LOGIT_STEP);
  q.slices = static_cast<int>(ceil_div(vocab, q.slice));
  const bool listed = tokens && history <= gws::LISTED;
  int64_t least = 0;
  for (int64_t blocks = ceil_div(q.slices, gws::MAX_LISTS); blocks < 2 * q.slices; blocks *= 2) {
    const int64_t each = ceil_div(q.slices, blocks);
    const int64_t slice = tokens && !listed ? 3 : 1, begin = tokens ? 3 : 1;
    const int64_t cost = ceil_div(rows * ceil_div(q.slices, each), held) * (each * slice + begin);
    if (q.each != 0 && cost >= least) continue;
    least = cost;
    q.each = static_cast<int>(each);
    q.blocks = static_cast<int>(ceil_div(q.slices, each));
  }
  q.shift = 0;
  while ((1 << q.shift) < q.slice) ++q.shift;
  q.lists = listed && q.each > 1;
  if (rows * q.blocks > kMaxDim) return GEMM_WS_ERR_INVALID_ARG;
  const size_t smem = 4 * ((tokens ? 2 * q.slice + 2 * q.slice / 32 : 0) +
                           (q.biases ? 2 * q.slice / 32 + 2 * q.biases : 0) + (q.lists ? gws::LISTED : 0));
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
