// Host side of the product of 8-bit integers (include/gemm_ws_lm.h): argument checks, the
// plan and the launches.
#include <cstring>

#include "lm_host.cuh"
#include "lm_int8_kernel.cuh"

namespace {

namespace i8 = gws::i8;

// A sum of this many products of two 8-bit integers fits 32 bits.
constexpr int64_t kMaxK = (int64_t{1} << 17) - 1;
// Extents whose last tile's rows stay in 32 bits.
constexpr int64_t kMaxExtent = (int64_t{1} << 31) - 4096;

template <int TOKENS>
int launch_dot(gemm_ws* h, i8::DotParams& q, cudaStream_t s) {
  const int64_t groups = ceil_div(q.channels, i8::DOT_ROWS);
  // as many warps for a group as leave each some of K, and more where there are few groups
  q.split = 1;
  while (q.split < i8::DOT_WARPS && groups * q.split < int64_t{16} * h->num_sms && q.k > 512 * q.split)
    q.split *= 2;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>(ceil_div(groups, i8::DOT_WARPS / q.split)),
                     static_cast<unsigned>(ceil_div(q.tokens, TOKENS)), 1);
  cfg.blockDim = dim3(i8::DOT_THREADS, 1, 1);
  cfg.stream = s;
  if (h->pdl) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  const cudaError_t e = cudaLaunchKernelEx(&cfg, i8::dot_kernel<TOKENS>, q);
  return e == cudaSuccess ? GEMM_WS_OK : cuda_fail(h, e);
}

}  // namespace

extern "C" {

int64_t gemm_ws_int8_matmul_workspace(gemm_ws_t* h, int64_t tokens, int64_t channels, int64_t k) {
  if (!h || tokens < 0 || channels < 1 || k < 1 || tokens > kMaxExtent || channels > kMaxExtent ||
      k > kMaxK || tokens * k > kMaxElems || channels * k > kMaxElems || tokens * channels > kMaxElems)
    return -GEMM_WS_ERR_INVALID_ARG;
  return 0;
}

int gemm_ws_int8_matmul(gemm_ws_t* h, const int8_t* a, int64_t lda, const float* a_scales,
                        const int8_t* w, int64_t ldw, const float* w_scales, const float* bias, void* d,
                        int64_t ldd, int dtype, int64_t tokens, int64_t channels, int64_t k,
                        void* workspace, int64_t workspace_bytes, void* stream) {
  const int64_t need = gemm_ws_int8_matmul_workspace(h, tokens, channels, k);
  if (need < 0 || dtype < GEMM_WS_BF16 || dtype > GEMM_WS_F32) return GEMM_WS_ERR_INVALID_ARG;
  if (tokens == 0) return GEMM_WS_OK;
  const Mat ma{a, lda, 1}, mw{w, ldw, 1}, md{d, ldd, element_size(dtype)};
  if (!a || !a_scales || !w || !w_scales || !d || bad_matrix(ma, k) || bad_matrix(mw, k) ||
      bad_matrix(md, channels) || (need > 0 && (!workspace || workspace_bytes < need)))
    return GEMM_WS_ERR_INVALID_ARG;
  for (const float* f : {a_scales, w_scales, bias})
    if (reinterpret_cast<uintptr_t>(f) % 4 != 0) return GEMM_WS_ERR_INVALID_ARG;
  if (!aligned16(w) || (channels > 1 && ldw % 16 != 0) || (need > 0 && reinterpret_cast<uintptr_t>(workspace) % 256 != 0))
    return GEMM_WS_ERR_ALIGNMENT;
  const Span outputs[] = {span(md, tokens, channels), {need > 0 ? workspace : nullptr, need}};
  const Span inputs[] = {span(ma, tokens, k), span(mw, channels, k), {a_scales, tokens * 4},
                         {w_scales, channels * 4}, {bias, channels * 4}};
  if (any_overlap(outputs, inputs)) return GEMM_WS_ERR_INVALID_ARG;
  DeviceGuard guard(h->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  i8::Output out;
  out.d = d;
  out.ldd = ldd;
  out.type = dtype;
  out.a_scales = a_scales;
  out.w_scales = w_scales;
  out.bias = bias;
  i8::DotParams q;
  std::memset(&q, 0, sizeof q);
  q.a = a;
  q.w = w;
  q.lda = lda;
  q.ldw = ldw;
  q.tokens = static_cast<int>(tokens);
  q.channels = static_cast<int>(channels);
  q.k = static_cast<int>(k);
  q.wide = aligned16(a) && (tokens == 1 || lda % 16 == 0);
  q.out = out;
  if (tokens <= 1) return launch_dot<1>(h, q, s);
  if (tokens <= 2) return launch_dot<2>(h, q, s);
  if (tokens <= 4) return launch_dot<4>(h, q, s);
  return launch_dot<8>(h, q, s);
}

}  // extern "C"
