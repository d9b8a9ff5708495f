// Host side of the product of 8-bit integers (include/gemm_ws_lm.h): argument checks, the
// plan and the launches.
#include <atomic>
#include <cstring>

#include "lm_host.cuh"
#include "lm_int8_kernel.cuh"
#ifdef GEMM_WS_DEBUG
#include "gemm_ws_debug.h"
#endif

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

// Up to four tokens the integer dot products of the CUDA cores keep up with w's bytes (4 tokens x
// 4096 over 131072: 102 us, by tensor cores 104; 8 tokens 188 and 104), and up to eight where w is so small
// that the tensor cores' start counts for more (8 x 4096 over 4096: 13 us and 14; 8 x 8192 over
// 8192: 40 and 24).
bool few(int64_t tokens, int64_t channels, int64_t k) {
  return tokens <= 4 || (tokens <= 8 && channels * k <= int64_t{1} << 24);
}

struct Plan {
  bool dot;
  int bn, splits;
  int64_t whole;     // tiles that are not cut
  int64_t tiles_m, tiles_n, stages, clusters;
  int64_t chunks;    // of 16 in a row of the tokens in fp16
  int64_t total, arrived;   // byte offsets in the workspace, behind the tokens in fp16
  int64_t bytes;            // of workspace
};

// Tiles as wide as leave the least work to the slowest pair: rounds times the time of a tile, where a
// stage of K takes as long as its MMAs, but no less than 128 tokens' (its conversion), and some more; and a
// tile's end as long as 3 stages, 7 where cuts of K are joined. Of the tiles of a last wave that do not reach
// all pairs K is cut (5000 x 4000 over 3000, 384 tiles for 76 pairs: 96 us, 113 with them whole).
Plan make_plan(const gemm_ws* h, int64_t tokens, int64_t channels, int64_t k) {
  Plan q;
  std::memset(&q, 0, sizeof q);
  q.dot = few(tokens, channels, k) || h->max_pair_clusters < 1;
  if (q.dot) return q;
  q.stages = ceil_div(k, i8::BK);
  q.tiles_n = ceil_div(channels, 2 * i8::BM);
  const int64_t pairs = h->max_pair_clusters;
  int64_t least = 0;
  for (int bn = i8::BN_MAX; bn >= 32; bn -= 32) {
    const int64_t tiles = ceil_div(tokens, bn) * q.tiles_n, rest = tiles % pairs;
    int64_t splits = rest ? pairs / rest : 1;
    if (splits > q.stages / 2) splits = q.stages / 2;   // at least 256 of K
    if (splits < 1 || q.stages + 3 <= ceil_div(q.stages, splits) + 7) splits = 1;
    const int64_t last = rest == 0 ? 0 : splits > 1 ? ceil_div(q.stages, splits) + 7 : q.stages + 3;
    const int64_t cost = (tiles / pairs * (q.stages + 3) + last) * ((bn > 128 ? bn : 128) + 32);
    if (q.bn != 0 && cost >= least) continue;
    least = cost;
    q.bn = bn;
    q.splits = static_cast<int>(splits);
    q.whole = splits > 1 ? tiles - rest : tiles;
  }
  q.tiles_m = ceil_div(tokens, q.bn);
  const int64_t cut = q.tiles_m * q.tiles_n - q.whole, units = q.whole + cut * q.splits;
  q.clusters = units < pairs ? units : pairs;
  q.chunks = ceil_div(k, 16);
  q.total = ceil_div(tokens * q.chunks * 32, 256) * 256;
  q.arrived = q.total + cut * 2 * q.bn * i8::BM * 4;
  q.bytes = q.arrived + ceil_div(cut * 2 * i8::EPI_WARPS * 4, 256) * 256;
  return q;
}

bool encode(gemm_ws* h, CUtensorMap* m, const void* ptr, bool half, int64_t inner, int64_t rows, int64_t ld,
            int x, int y) {
  const int64_t size = half ? 2 : 1;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows), 1};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld * size), static_cast<cuuint64_t>(ld * rows * size)};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(x), static_cast<cuuint32_t>(y), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = h->encode(
      m, half ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(ptr),
      dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
      CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) h->last_cuda_error = static_cast<int>(r);
  return r == CUDA_SUCCESS;
}

// Whether the product kernel has the registers at launch that its warpgroups share out: with fewer
// they would wait for each other forever. (A property of the built kernel.)
bool registers_as_planned(const gemm_ws* h) {
#ifdef GEMM_WS_DEBUG
  if (h->debug_fault == 6) return false;   // injected fault
#endif
  (void)h;
  static std::atomic<bool> seen{false};   // handles may be used by several threads
  if (seen.load(std::memory_order_relaxed)) return true;
  cudaFuncAttributes a;
  if (cudaFuncGetAttributes(&a, i8::product_kernel) != cudaSuccess || a.numRegs != i8::REGS_LAUNCH) return false;
  seen.store(true, std::memory_order_relaxed);
  return true;
}

int launch_product(gemm_ws* h, const Plan& q, const i8::Params& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  cfg.gridDim = dim3(static_cast<unsigned>(2 * q.clusters), 1, 1);
  cfg.blockDim = dim3(i8::THREADS, 1, 1);
  cfg.dynamicSmemBytes = i8::SMEM_BYTES;
  cfg.stream = s;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = h->pdl ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, i8::product_kernel, p);
  return e == cudaSuccess ? GEMM_WS_OK : cuda_fail(h, e);
}

}  // namespace

extern "C" {

int64_t gemm_ws_int8_matmul_workspace(gemm_ws_t* h, int64_t tokens, int64_t channels, int64_t k) {
  if (!h || tokens < 0 || channels < 1 || k < 1 || tokens > kMaxExtent || channels > kMaxExtent ||
      k > kMaxK || tokens * k > kMaxElems || channels * k > kMaxElems || tokens * channels > kMaxElems)
    return -GEMM_WS_ERR_INVALID_ARG;
  return tokens == 0 ? 0 : make_plan(h, tokens, channels, k).bytes;
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
      bad_matrix(md, channels) || ldw > kMaxElems / channels || (need > 0 && (!workspace || workspace_bytes < need)))
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
  out.channels = static_cast<int>(channels);
  out.pairs = reinterpret_cast<uintptr_t>(d) % 4 == 0 && (tokens == 1 || ldd % 2 == 0);
  out.a_scales = a_scales;
  out.w_scales = w_scales;
  out.bias = bias;
  const bool wide = aligned16(a) && (tokens == 1 || lda % 16 == 0);
  const Plan plan = make_plan(h, tokens, channels, k);
  if (plan.dot) {
    i8::DotParams q;
    std::memset(&q, 0, sizeof q);
    q.a = a;
    q.w = w;
    q.lda = lda;
    q.ldw = ldw;
    q.tokens = static_cast<int>(tokens);
    q.channels = static_cast<int>(channels);
    q.k = static_cast<int>(k);
    q.wide = wide;
    q.out = out;
    if (tokens <= 1) return launch_dot<1>(h, q, s);
    if (tokens <= 2) return launch_dot<2>(h, q, s);
    if (tokens <= 4) return launch_dot<4>(h, q, s);
    return launch_dot<8>(h, q, s);
  }
  // What may be refused is, before anything is launched.
  if (!registers_as_planned(h)) return GEMM_WS_ERR_BUILD;
  const cudaError_t allowed = allow_smem(h, reinterpret_cast<const void*>(i8::product_kernel), i8::SMEM_BYTES);
  if (allowed != cudaSuccess) return cuda_fail(h, allowed);
  i8::ExpandParams e;
  std::memset(&e, 0, sizeof e);
  e.a = a;
  e.lda = lda;
  e.tokens = static_cast<int>(tokens);
  e.k = static_cast<int>(k);
  e.wide = wide;
  e.chunks = static_cast<int>(plan.chunks);
  e.out = static_cast<uint16_t*>(workspace);
  e.zero = reinterpret_cast<uint4*>(static_cast<uint8_t*>(workspace) + plan.total);
  e.zeros = (plan.bytes - plan.total) / 16;
  i8::Params q;
  std::memset(&q, 0, sizeof q);
  const int64_t pitch = 16 * plan.chunks;
  if (!encode(h, &q.tmW, w, false, k, channels, channels > 1 ? ldw : ceil_div(k, 16) * 16, i8::BK, i8::BM) ||
      !encode(h, &q.tmA, workspace, true, pitch, tokens, pitch, i8::HALF_K, plan.bn / 2))
    return GEMM_WS_ERR_CUDA;
  const int rc = launch(h, i8::expand_kernel, ceil_div(tokens * plan.chunks + e.zeros, i8::EXPAND_THREADS),
                        i8::EXPAND_THREADS, 0, s, e);
  if (rc != GEMM_WS_OK) return rc;
  q.tokens = static_cast<int>(tokens);
  q.channels = static_cast<int>(channels);
  q.stages = static_cast<int>(plan.stages);
  q.bn = plan.bn;
  const i8::Rings rings = i8::rings_of(q.bn);
  q.bufs = rings.bufs;
  q.a_stages = rings.a_stages;
  q.w_stages = rings.w_stages;
  q.tiles_m = static_cast<int>(plan.tiles_m);
  q.tiles_n = static_cast<int>(plan.tiles_n);
  q.whole = static_cast<int>(plan.whole);
  q.splits = plan.splits;
  q.total = reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + plan.total);
  q.arrived = reinterpret_cast<uint32_t*>(static_cast<uint8_t*>(workspace) + plan.arrived);
  q.out = out;
  q.status = h->work + 1;
  q.timeout_ns = h->timeout_ns;
#ifdef GEMM_WS_DEBUG
  q.debug_fault = h->debug_fault;
#endif
  return launch_product(h, plan, q, s);
}

#ifdef GEMM_WS_DEBUG
int gemm_ws_debug_int8_rings(int bn, int* rings) {
  if (bn < 32 || bn > i8::BN_MAX || bn % 32 != 0 || !rings) return GEMM_WS_ERR_INVALID_ARG;
  const i8::Rings r = i8::rings_of(bn);
  rings[0] = r.bufs;
  rings[1] = r.w_stages;
  rings[2] = r.a_stages;
  rings[3] = i8::T_FULL_ARRIVALS;
  rings[4] = i8::CONV_WARPS;
  rings[5] = i8::CUT_STAGES;
  return GEMM_WS_OK;
}
#endif

}  // extern "C"
