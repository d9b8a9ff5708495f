// Host side of the linear cross entropy (include/gemm_ws_lm.h): argument
// checks, the plan (tiles, pieces of the vocabulary, cuts of K), the workspace's
// layout, tensor maps and launches.
#include <cstring>

#include "gemm_ws_lm.h"
#ifdef GEMM_WS_DEBUG
#include "gemm_ws_debug.h"
#endif
#include "handle.cuh"
#include "lm_loss_kernel.cuh"

namespace {

namespace ce = gws::ce;

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
int64_t round_up(int64_t a, int64_t b) { return ceil_div(a, b) * b; }

// The tiles of one launch.
struct Tiling {
  int cg, bn;
  int64_t clusters;   // that run at once
};

// CTA pairs with 256 x 256 tiles where they make a full wave; else single
// CTAs with the tile width that leaves the least work to the slowest one
// (rounds times columns, and 64 columns' worth of time a round for the tile's
// rows and hand-over). Up to 128 rows a pair's second CTA would idle.
// `step`: what the width must be a multiple of.
Tiling pick_tiling(const gemm_ws* h, int64_t m, int64_t n, int step) {
  // as many as of the GEMM's: both have one CTA on an SM
  const int64_t pairs = h->max_pair_clusters;
  if (pairs > 0 && m > ce::BM && ceil_div(m, 2 * ce::BM) * ceil_div(n, ce::BN_MAX) >= pairs)
    return {2, ce::BN_MAX, pairs};
  Tiling best = {1, ce::BN_MAX, h->num_sms};
  int64_t least = 0;
  for (int bn = ce::BN_MAX; bn >= 64; bn -= step) {
    const int64_t cost =
        ceil_div(ceil_div(m, ce::BM) * ceil_div(n, bn), h->num_sms) * (bn + 64);
    if (bn == ce::BN_MAX || cost < least) {
      least = cost;
      best.bn = bn;
    }
  }
  return best;
}

// G of one piece, in whole tiles of rows, takes at most this many bytes, or 4096 columns.
constexpr int64_t kPieceBytes = int64_t{256} << 20;
constexpr int64_t kMinPiece = 4096;
constexpr int64_t kShortK = 128;
// dx's sums are cut along the vocabulary where its tiles alone do not fill the GPU.
constexpr int64_t kMaxCuts = 16;

struct Plan {
  Tiling logits;      // forward: all of the vocabulary; backward: a piece
  Tiling sums;
  int carry;
  int64_t slots;      // partial maxima and sums a row
  int64_t piece, pieces;
  int64_t cuts;
  int64_t pitch, rows;   // of the packed rows of x; rows of G, too
  int64_t blocks;     // of the joining kernel
  // byte offsets in the workspace
  int64_t packed, place, target, count, logit, part, block_sum, lse, grad, scale, g, sums_at,
      bytes;
};

Plan make_plan(const gemm_ws* h, int64_t T, int64_t H, int64_t V, bool backward) {
  Plan q;
  std::memset(&q, 0, sizeof q);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += round_up(bytes, 256);
    return here;
  };
  q.pitch = round_up(H, 64);   // whole 128-byte lines: x's boxes never straddle one
  // Whole tiles of rows (they may hold anything past the counted ones): the TMA
  // fills rows that are not there more slowly than it fetches rows that are.
  q.rows = T > ce::BM ? round_up(T, 2 * ce::BM) : ce::BM;
  q.packed = take(q.rows * q.pitch * 2);
  q.place = take(T * 4);
  q.target = take(T * 4);
  q.count = take(4);
  if (!backward) {
    q.logits = pick_tiling(h, T, V, 32);
    q.carry = T <= ce::BM;
    const int64_t tiles_n = ceil_div(V, q.logits.bn);
    q.slots = 2 * (q.carry && tiles_n > q.logits.clusters ? q.logits.clusters : tiles_n);
    q.blocks = ceil_div(T, ce::JOIN_ROWS);
    q.logit = take(T * 4);
    q.part = take(q.slots * T * 8);
    q.block_sum = take(q.blocks * 4);
  } else {
    q.piece = kPieceBytes / (2 * q.rows) / ce::BN_MAX * ce::BN_MAX;
    if (q.piece < kMinPiece) q.piece = kMinPiece;
    if (q.piece > round_up(V, ce::BN_MAX)) q.piece = round_up(V, ce::BN_MAX);
    q.pieces = ceil_div(V, q.piece);
    q.piece = round_up(ceil_div(V, q.pieces), ce::BN_MAX);   // about equal
    q.pieces = ceil_div(V, q.piece);
    q.logits = pick_tiling(h, T, q.piece, 64);
    // dx has ceil(T / 128) x ceil(H / bn) tiles, dweight piece / 128 times
    // ceil(H / bn); both run in one launch.
    const int64_t rows = T + q.piece;
    q.sums = pick_tiling(h, rows, H, 64);
    // dweight's K is the tokens. Where that is short its tiles' stores bound the
    // launch, which single CTAs do better (4096 hidden over 32768, both gradients: 128
    // tokens 171 us against 222 with pairs; 200 tokens 220 against 216).
    if (T <= kShortK) q.sums = {1, ce::BN_MAX, h->num_sms};
    const int64_t tiles = ceil_div(T, ce::BM * q.sums.cg) * ceil_div(H, q.sums.bn);
    const int64_t stages = ceil_div(q.piece, ce::BK * q.sums.cg);
    q.cuts = tiles < q.sums.clusters ? q.sums.clusters / tiles : 1;
    if (q.cuts > stages / 4) q.cuts = stages / 4 > 0 ? stages / 4 : 1;
    if (q.cuts > kMaxCuts) q.cuts = kMaxCuts;
    q.lse = take(T * 4);
    q.grad = take(T * 4);
    q.scale = take(4);
    q.g = take(q.rows * q.piece * 2);
    q.sums_at = take(q.cuts * T * H * 4);
  }
  q.bytes = at;
  return q;
}

// A tensor of `depth` slices of `rows` rows of `inner` contiguous elements;
// box x by y.
bool encode(gemm_ws* h, CUtensorMap* m, const void* ptr, bool f32, int64_t inner, int64_t rows,
            int64_t depth, int64_t ld, int64_t slice, int x, int y) {
  const int64_t size = f32 ? 4 : 2;
  cuuint64_t dims[3] = {static_cast<cuuint64_t>(inner), static_cast<cuuint64_t>(rows),
                        static_cast<cuuint64_t>(depth)};
  cuuint64_t strides[2] = {static_cast<cuuint64_t>(ld * size), static_cast<cuuint64_t>(slice * size)};
  cuuint32_t box[3] = {static_cast<cuuint32_t>(x), static_cast<cuuint32_t>(y), 1};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUresult r = h->encode(
      m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
      const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
      CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) h->last_cuda_error = static_cast<int>(r);
  return r == CUDA_SUCCESS;
}

// An operand of a product: rows of `inner` bf16, K or MN contiguous.
bool operand(gemm_ws* h, CUtensorMap* m, const void* ptr, int64_t inner, int64_t rows, int64_t ld,
             bool mn, int box_rows) {
  return encode(h, m, ptr, false, inner, rows, 1, ld, ld * rows, 64, mn ? 64 : box_rows);
}

// Rows of x in a box: fewer than 128 tokens come in a box of their own size. (One
// token over 131072 x 4096 took 238 us with boxes of 128 rows, of which 127 were
// not there; now 172.)
int box_rows(int64_t T) { return static_cast<int>(T < ce::BM ? T : ce::BM); }

template <typename P>
int launch(gemm_ws* h, void (*kernel)(P), int64_t blocks, int threads, size_t smem, int cluster,
           cudaStream_t s, const P& params) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  int n = 0;
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  if (h->pdl) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  if (cluster > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  cudaError_t e = cudaSuccess;
  if (smem > kDefaultSmem) e = allow_smem(h, reinterpret_cast<const void*>(kernel), smem);
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kernel, params);
  return e == cudaSuccess ? GEMM_WS_OK : cuda_fail(h, e);
}

// One persistent product launch; `units`: at most how many units it has.
template <int MODE>
int launch_product(gemm_ws* h, const Tiling& t, int64_t units, const ce::Params& p, cudaStream_t s) {
  const int64_t clusters = units < t.clusters ? units : t.clusters;
  if (t.cg == 2)
    return launch(h, ce::product_kernel<2, MODE>, 2 * clusters, ce::THREADS, ce::SMEM_BYTES, 2, s, p);
  return launch(h, ce::product_kernel<1, MODE>, clusters, ce::THREADS, ce::SMEM_BYTES, 1, s, p);
}

int ring_stages(const Tiling& t) {
  const uint32_t bytes = t.cg == 2 ? ce::stage_bytes<2>(t.bn) : ce::stage_bytes<1>(t.bn);
  const int n = static_cast<int>(ce::RING_BYTES / bytes);
  return n < ce::MAX_STAGES ? n : ce::MAX_STAGES;
}

// Rows, columns and the copies' coordinates are 32-bit numbers in the kernels, up to
// the end of an extent's last tile, stage or piece, which lies less than this far behind it.
constexpr int64_t kMaxExtent = (int64_t{1} << 31) - 4096;

int check_sizes(const gemm_ws* h, int64_t T, int64_t H, int64_t V) {
  if (!h || T < 0 || H < 1 || V < 1 || T > kMaxExtent || H > kMaxExtent || V > kMaxExtent)
    return GEMM_WS_ERR_INVALID_ARG;
  if (T * H > kMaxElems || V * H > kMaxElems || T * V > kMaxElems) return GEMM_WS_ERR_INVALID_ARG;
  if (H % 8 != 0) return GEMM_WS_ERR_ALIGNMENT;
  return GEMM_WS_OK;
}

struct Span {
  const void* ptr;
  int64_t bytes;
};

// Whether one of the outputs overlaps another one or an input.
bool any_overlap(const Span* out, int outs, const Span* in, int ins) {
  for (int i = 0; i < outs; ++i) {
    for (int j = i + 1; j < outs; ++j)
      if (overlaps(out[i].ptr, out[i].bytes, out[j].ptr, out[j].bytes)) return true;
    for (int j = 0; j < ins; ++j)
      if (overlaps(out[i].ptr, out[i].bytes, in[j].ptr, in[j].bytes)) return true;
  }
  return false;
}

int64_t matrix_bytes(int64_t rows, int64_t cols, int64_t ld) { return 2 * ((rows - 1) * ld + cols); }

bool odd(const void* p, int64_t to) { return reinterpret_cast<uintptr_t>(p) % to != 0; }

// What both directions ask of their common arguments.
int check_common(const gemm_ws* h, const uint16_t* x, int64_t ldx, const uint16_t* weight,
                 int64_t ldw, const void* target, int target_bytes, int64_t T, int64_t H,
                 int64_t V) {
  const int rc = check_sizes(h, T, H, V);
  if (rc != GEMM_WS_OK) return rc;
  if (target_bytes != 4 && target_bytes != 8) return GEMM_WS_ERR_INVALID_ARG;
  if (T > 0 && (!x || !target || ldx < H || ldx > kMaxElems || odd(x, 2) || odd(target, target_bytes)))
    return GEMM_WS_ERR_INVALID_ARG;
  if (T > 0 && (!weight || ldw < H || ldw > kMaxElems)) return GEMM_WS_ERR_INVALID_ARG;
  if (T > 0 && (odd(weight, 16) || ldw % 8 != 0)) return GEMM_WS_ERR_ALIGNMENT;
  return GEMM_WS_OK;
}

ce::Targets targets(const void* target, int target_bytes, int64_t ignore, int64_t V) {
  return {target, target_bytes == 8, ignore, static_cast<int>(V)};
}

ce::PackParams pack_params(const Plan& q, uint8_t* ws, const uint16_t* x, int64_t ldx,
                           const void* target, int target_bytes, int64_t ignore, int64_t T,
                           int64_t H, int64_t V, int num_sms) {
  ce::PackParams p;
  std::memset(&p, 0, sizeof p);
  p.x = x;
  p.ldx = ldx;
  p.given = targets(target, target_bytes, ignore, V);
  p.rows = static_cast<int>(T);
  p.cols = static_cast<int>(H);
  p.wide = !odd(x, 16) && ldx % 8 == 0;
  p.padded = static_cast<int>(round_up(T, 128));
  int64_t chunk = ceil_div(p.padded, int64_t{8} * num_sms);
  p.chunk = static_cast<int>(chunk < ce::PACK_THREADS ? chunk : ce::PACK_THREADS);
  p.packed = reinterpret_cast<uint16_t*>(ws + q.packed);
  p.pitch = q.pitch;
  p.place = reinterpret_cast<int*>(ws + q.place);
  p.target_out = reinterpret_cast<int*>(ws + q.target);
  p.count = reinterpret_cast<int*>(ws + q.count);
  return p;
}

ce::Params product_params(const gemm_ws* h, const Plan& q, uint8_t* ws, const Tiling& t, int64_t T) {
  ce::Params p;
  std::memset(&p, 0, sizeof p);
  p.jobs = 1;
  p.bn = t.bn;
  p.stages = ring_stages(t);
  p.a_rows = ce::BM;
  p.cut_k = T <= ce::BM ? ce::CUT_K_FEW : ce::CUT_K;
  p.count = reinterpret_cast<const int*>(ws + q.count);
  p.target = reinterpret_cast<const int*>(ws + q.target);
  p.part_stride = T;
  p.status = h->work + 1;
  p.timeout_ns = h->timeout_ns;
#ifdef GEMM_WS_DEBUG
  p.debug_fault = h->debug_fault;
#endif
  return p;
}

}  // namespace

extern "C" {

int64_t gemm_ws_linear_ce_workspace(gemm_ws_t* h, int64_t tokens, int64_t hidden, int64_t vocab,
                                    int backward) {
  const int rc = check_sizes(h, tokens, hidden, vocab);
  if (rc != GEMM_WS_OK) return -rc;
  return tokens == 0 ? 0 : make_plan(h, tokens, hidden, vocab, backward != 0).bytes;
}

int gemm_ws_linear_ce(gemm_ws_t* h, const uint16_t* x, int64_t ldx, const uint16_t* weight,
                      int64_t ldw, const void* target, int target_bytes, int64_t ignore,
                      float* loss, float* lse, float* mean, int64_t tokens, int64_t hidden,
                      int64_t vocab, void* workspace, int64_t workspace_bytes, void* stream) {
  const int64_t T = tokens, H = hidden, V = vocab;
  int rc = check_common(h, x, ldx, weight, ldw, target, target_bytes, T, H, V);
  if (rc != GEMM_WS_OK) return rc;
  if (odd(mean, 4)) return GEMM_WS_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (T == 0) {
    if (!mean) return GEMM_WS_OK;
    DeviceGuard guard(h->device);
    const cudaError_t e = cudaMemsetAsync(mean, 0, 8, s);
    return e == cudaSuccess ? GEMM_WS_OK : cuda_fail(h, e);
  }
  if (!loss || !lse || odd(loss, 4) || odd(lse, 4)) return GEMM_WS_ERR_INVALID_ARG;
  const Plan q = make_plan(h, T, H, V, false);
  if (!workspace || workspace_bytes < q.bytes) return GEMM_WS_ERR_INVALID_ARG;
  if (odd(workspace, 256)) return GEMM_WS_ERR_ALIGNMENT;
  const Span out[4] = {{loss, 4 * T}, {lse, 4 * T}, {mean, 8}, {workspace, q.bytes}};
  const Span in[3] = {{x, matrix_bytes(T, H, ldx)}, {weight, matrix_bytes(V, H, ldw)},
                      {target, target_bytes * T}};
  if (any_overlap(out, 4, in, 3)) return GEMM_WS_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);

  ce::PackParams pack = pack_params(q, ws, x, ldx, target, target_bytes, ignore, T, H, V, h->num_sms);
  pack.target_logit = reinterpret_cast<float*>(ws + q.logit);

  ce::Params p = product_params(h, q, ws, q.logits, T);
  ce::Job& job = p.job[0];
  job.m = -1;
  job.n = static_cast<int>(V);
  job.k = static_cast<int>(H);
  job.splits = 1;
  job.out = ce::OUT_LSE;
  p.a_rows = box_rows(T);
  p.cols = static_cast<int>(V);
  p.target_logit = pack.target_logit;
  p.part = reinterpret_cast<float2*>(ws + q.part);
  p.carry = q.carry;
  p.slots = static_cast<int>(q.slots);
  p.result = {loss, lse, mean};
  p.done = h->work + 3;
  const int64_t units = ceil_div(T, ce::BM * q.logits.cg) * ceil_div(V, q.logits.bn);
  if (!operand(h, &job.tmB, weight, H, V, ldw, false, q.logits.bn / q.logits.cg))
    return GEMM_WS_ERR_CUDA;
  DeviceGuard guard(h->device);

  // Rows that the TMA can read where they lie are not packed if there are up to 128 of
  // them, or if all tiles run at once, so that packing could save none of their time:
  // each row has its own sums, so an uncounted one touches nothing. (256 x 256 over 1000
  // words 10.3 us, packed 12.3; 2100 x 1024 over 1000 15.5 and 19.7.)
  p.direct = pack.wide && (T <= ce::BM || units <= q.logits.clusters);
  p.join = p.direct && T <= ce::JOIN_FEW;
  p.rows = static_cast<int>(T);
  p.given = pack.given;
  if (!(p.direct ? operand(h, &job.tmA, x, H, T, ldx, false, p.a_rows)
                 : operand(h, &job.tmA, pack.packed, H, q.rows, q.pitch, false, p.a_rows)))
    return GEMM_WS_ERR_CUDA;
  rc = GEMM_WS_OK;
  if (!p.direct)
    rc = launch(h, ce::pack_kernel, ceil_div(pack.padded, pack.chunk), ce::PACK_THREADS, 0, 1, s, pack);
  if (rc == GEMM_WS_OK) rc = launch_product<ce::LSE>(h, q.logits, units, p, s);
  if (rc != GEMM_WS_OK || p.join) return rc;

  ce::JoinParams join;
  std::memset(&join, 0, sizeof join);
  join.part = p.part;
  join.part_stride = T;
  join.slots = p.slots;
  join.direct = p.direct;
  join.given = p.given;
  join.place = pack.place;
  join.count = pack.count;
  join.target_logit = pack.target_logit;
  join.rows = static_cast<int>(T);
  join.result = p.result;
  join.block_sum = reinterpret_cast<float*>(ws + q.block_sum);
  join.done = p.done;
  return launch(h, ce::join_kernel, q.blocks, ce::JOIN_ROWS * ce::JOIN_LANES, 0, 1, s, join);
}

int gemm_ws_linear_ce_backward(gemm_ws_t* h, const uint16_t* x, int64_t ldx,
                               const uint16_t* weight, int64_t ldw, const void* target,
                               int target_bytes, int64_t ignore, const float* lse,
                               const float* grad, int grad_step, uint16_t* dx, int64_t lddx,
                               uint16_t* dweight, int64_t lddw, int64_t tokens, int64_t hidden,
                               int64_t vocab, void* workspace, int64_t workspace_bytes,
                               void* stream) {
  const int64_t T = tokens, H = hidden, V = vocab;
  int rc = check_common(h, x, ldx, weight, ldw, target, target_bytes, T, H, V);
  if (rc != GEMM_WS_OK) return rc;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if ((dweight && (lddw < H || lddw > kMaxElems)) || (dx && (lddx < H || lddx > kMaxElems)) ||
      (grad_step != 0 && grad_step != 1))
    return GEMM_WS_ERR_INVALID_ARG;
  if (odd(dweight, 16) || odd(dx, 16) || (dweight && lddw % 8 != 0) || (dx && lddx % 8 != 0))
    return GEMM_WS_ERR_ALIGNMENT;
  if (T == 0) {
    if (!dweight) return GEMM_WS_OK;
    DeviceGuard guard(h->device);
    const cudaError_t e = cudaMemset2DAsync(dweight, 2 * lddw, 0, 2 * H, V, s);
    return e == cudaSuccess ? GEMM_WS_OK : cuda_fail(h, e);
  }
  if (!lse || !grad || odd(lse, 4) || odd(grad, 4)) return GEMM_WS_ERR_INVALID_ARG;
  if (!dx && !dweight) return GEMM_WS_OK;
  const Plan q = make_plan(h, T, H, V, true);
  if (!workspace || workspace_bytes < q.bytes) return GEMM_WS_ERR_INVALID_ARG;
  if (odd(workspace, 256)) return GEMM_WS_ERR_ALIGNMENT;
  const Span out[3] = {{dx, dx ? matrix_bytes(T, H, lddx) : 0},
                       {dweight, dweight ? matrix_bytes(V, H, lddw) : 0},
                       {workspace, q.bytes}};
  const Span in[5] = {{x, matrix_bytes(T, H, ldx)}, {weight, matrix_bytes(V, H, ldw)},
                      {target, target_bytes * T}, {lse, 4 * T}, {grad, grad_step ? 4 * T : 4}};
  if (any_overlap(out, 3, in, 5)) return GEMM_WS_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);

  ce::PackParams pack = pack_params(q, ws, x, ldx, target, target_bytes, ignore, T, H, V, h->num_sms);
  pack.lse = lse;
  pack.grad = grad;
  pack.grad_step = grad_step;
  pack.lse_out = reinterpret_cast<float*>(ws + q.lse);
  pack.grad_out = reinterpret_cast<float*>(ws + q.grad);
  pack.scale = reinterpret_cast<float*>(ws + q.scale);
  uint16_t* g = reinterpret_cast<uint16_t*>(ws + q.g);
  float* sums = reinterpret_cast<float*>(ws + q.sums_at);

  // The products of a piece; what changes from piece to piece is set below.
  ce::Params pg = product_params(h, q, ws, q.logits, T);
  pg.a_rows = box_rows(T);
  pg.lse = pack.lse_out;
  pg.grad = pack.grad_out;
  ce::Job& jg = pg.job[0];
  jg.m = -1;
  jg.k = static_cast<int>(H);
  jg.splits = 1;
  jg.out = ce::OUT_GRAD;
  ce::Params ps = product_params(h, q, ws, q.sums, T);
  ps.jobs = 0;
  ps.scale = pack.scale;
  const int b_rows = q.sums.bn / q.sums.cg;
  ce::Job* jx = dx ? &ps.job[ps.jobs++] : nullptr;
  ce::Job* jw = dweight ? &ps.job[ps.jobs++] : nullptr;
  bool ok = operand(h, &jg.tmA, pack.packed, H, q.rows, q.pitch, false, pg.a_rows) &&
            operand(h, &jg.tmB, weight, H, V, ldw, false, q.logits.bn / q.logits.cg);
  if (jx) {
    jx->m = -1;
    jx->n = static_cast<int>(H);
    jx->b_mn = 1;
    jx->splits = static_cast<int>(q.cuts);
    jx->out = ce::OUT_ADD;
    ok = ok && operand(h, &jx->tmB, weight, H, V, ldw, true, b_rows) &&
         encode(h, &jx->tmD, sums, true, H, T, q.cuts, H, T * H, 32, 32);
  }
  if (jw) {
    jw->n = static_cast<int>(H);
    jw->k = -1;
    jw->a_mn = jw->b_mn = 1;
    jw->splits = 1;
    jw->out = ce::OUT_BF16;
    ok = ok && operand(h, &jw->tmB, pack.packed, H, q.rows, q.pitch, true, b_rows) &&
         encode(h, &jw->tmD, dweight, false, H, V, 1, lddw, lddw * V, 64, 32);
  }
  if (!ok) return GEMM_WS_ERR_CUDA;

  DeviceGuard guard(h->device);
  rc = launch(h, ce::pack_kernel, ceil_div(pack.padded, pack.chunk), ce::PACK_THREADS, 0, 1, s, pack);
  for (int64_t i = 0; i < q.pieces && rc == GEMM_WS_OK; ++i) {
    const int64_t c0 = i * q.piece, cols = V - c0 < q.piece ? V - c0 : q.piece;
    const int64_t held = round_up(cols, 8);   // G's columns of this piece; the last few may be zeros
    jg.n = static_cast<int>(cols);
    jg.b_row0 = static_cast<int>(c0);
    pg.cols = static_cast<int>(cols);
    pg.col0 = static_cast<int>(c0);
    ok = encode(h, &jg.tmD, g, false, held, q.rows, 1, q.piece, q.piece * q.rows, 64, 32);
    int64_t units = 0;
    if (jx) {
      jx->k = static_cast<int>(cols);
      jx->b_row0 = static_cast<int>(c0);
      jx->add = i > 0;
      units += ceil_div(T, ce::BM * q.sums.cg) * ceil_div(H, q.sums.bn) * q.cuts;
      ok = ok && operand(h, &jx->tmA, g, held, q.rows, q.piece, false, ce::BM);
    }
    if (jw) {
      jw->m = static_cast<int>(cols);
      jw->d_row0 = static_cast<int>(c0);
      units += ceil_div(cols, ce::BM * q.sums.cg) * ceil_div(H, q.sums.bn);
      ok = ok && operand(h, &jw->tmA, g, held, q.rows, q.piece, true, ce::BM);
    }
    if (!ok) return GEMM_WS_ERR_CUDA;
    rc = launch_product<ce::GRAD>(
        h, q.logits, ceil_div(T, ce::BM * q.logits.cg) * ceil_div(cols, q.logits.bn), pg, s);
    if (rc == GEMM_WS_OK) rc = launch_product<ce::SUMS>(h, q.sums, units, ps, s);
  }
  if (rc == GEMM_WS_OK && dx) {
    ce::SpreadParams sp;
    std::memset(&sp, 0, sizeof sp);
    sp.sums = sums;
    sp.cuts = static_cast<int>(q.cuts);
    sp.cut_stride = T * H;
    sp.place = pack.place;
    sp.grad = pack.grad_out;
    sp.scale = pack.scale;
    sp.rows = static_cast<int>(T);
    sp.cols = static_cast<int>(H);
    sp.dx = dx;
    sp.lddx = lddx;
    rc = launch(h, ce::spread_kernel, ceil_div(T * (H / 4), ce::SPREAD_THREADS), ce::SPREAD_THREADS,
                0, 1, s, sp);
  }
  return rc;
}

#ifdef GEMM_WS_DEBUG
}  // extern "C"

namespace {

template <int CG>
int64_t list_units(const ce::Params& p, int count, int clusters, int* rows, int64_t max_rows) {
  int64_t n = 0;
  for (int c = 0; c < clusters; ++c) {
    const ce::Walk walk = ce::make_walk<CG>(p, count, c, clusters);
    ce::Unit w;
    for (int i = 0; ce::next_unit<CG>(p, walk, i, w); ++i, ++n) {
      if (n >= max_rows) continue;
      int* r = rows + n * 8;
      r[0] = c;
      r[1] = i;
      r[2] = static_cast<int>(w.job - p.job);
      r[3] = w.m0;
      r[4] = w.n0;
      r[5] = w.cut;
      r[6] = w.s0;
      r[7] = w.s1;
    }
  }
  return n;
}

}  // namespace

extern "C" {

int gemm_ws_debug_ce_units(int cta_group, int clusters, int bn, int count, const int* jobs,
                           int num_jobs, int* rows, int64_t max_rows, int64_t* num_rows) {
  if (cta_group < 1 || cta_group > 2 || clusters < 1 || bn < 16 || count < 0 || !jobs ||
      num_jobs < 1 || num_jobs > 2 || !num_rows)
    return GEMM_WS_ERR_INVALID_ARG;
  ce::Params p;
  std::memset(&p, 0, sizeof p);
  p.jobs = num_jobs;
  p.bn = bn;
  for (int j = 0; j < num_jobs; ++j) {
    p.job[j].m = jobs[4 * j];
    p.job[j].n = jobs[4 * j + 1];
    p.job[j].k = jobs[4 * j + 2];
    p.job[j].splits = jobs[4 * j + 3];
  }
  *num_rows = cta_group == 2 ? list_units<2>(p, count, clusters, rows, rows ? max_rows : 0)
                             : list_units<1>(p, count, clusters, rows, rows ? max_rows : 0);
  return GEMM_WS_OK;
}
#endif

}  // extern "C"
