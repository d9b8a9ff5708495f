// Host side of dropout and the norm (include/gemm_ws_lm.h): argument checks,
// the choice of a row's team of threads, and the launches.
#include <cmath>
#include <cstring>

#include "gemm_ws_lm.h"
#ifdef GEMM_WS_DEBUG
#include "gemm_ws_debug.h"
#endif
#include "handle.cuh"
#include "lm_norm_kernel.cuh"

namespace {

constexpr int64_t kMaxCols = 1024 * gws::MAX_VPT * gws::GROUP;   // 32768: a block holds a row
// fp32 partials of the handle: one row of kMaxCols for each SM.
constexpr int64_t kPartialPerSm = int64_t{128} * 256;
static_assert(kPartialPerSm >= kMaxCols, "a block's dweight partial fits its SM's share");

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

int element_size(int dtype) { return dtype == GEMM_WS_F32 ? 4 : 2; }

// A matrix argument as the checks see it.
struct Mat {
  const void* ptr;
  int64_t ld;
  int64_t size;   // bytes of an element
  bool given() const { return ptr != nullptr; }
  int64_t bytes(int64_t rows, int64_t cols) const { return ((rows - 1) * ld + cols) * size; }
  // Each row starts on a boundary of 8 elements (16 bytes at most).
  bool wide() const {
    const int64_t step = size * 8 < 16 ? size * 8 : 16;
    return reinterpret_cast<uintptr_t>(ptr) % step == 0 && (ld * size) % step == 0;
  }
};

// The output `out` may be exactly the input `in`, and else not overlap it.
bool clash(const Mat& out, const Mat& in, int64_t rows, int64_t cols, bool may_equal) {
  if (!out.given() || !in.given()) return false;
  if (may_equal && out.ptr == in.ptr && out.ld == in.ld && out.size == in.size) return false;
  return overlaps(out.ptr, out.bytes(rows, cols), in.ptr, in.bytes(rows, cols));
}

bool bad_matrix(const Mat& m, int64_t cols) {
  return m.given() && (m.ld < cols || m.ld > kMaxElems ||
                       reinterpret_cast<uintptr_t>(m.ptr) % m.size != 0);
}

// p and rng as a launch takes them. Returns false where p is not in [0, 1] or
// a mask is wanted and rng is missing.
bool make_dropout(const gemm_ws* h, double p, const uint64_t* rng, gws::Dropout* d) {
  if (!(p >= 0.0 && p <= 1.0)) return false;
  const int64_t below = static_cast<int64_t>(std::nearbyint(p * 65536.0));
  d->on = below > 0;
  d->rng = d->on ? rng : reinterpret_cast<const uint64_t*>(h->work);
  d->limit = static_cast<uint32_t>((below << 16) - 1);
  d->scale = below < 65536 ? static_cast<float>(65536.0 / (65536 - below)) : 0.0f;
  return !d->on || (rng && reinterpret_cast<uintptr_t>(rng) % 8 == 0);
}

// A launch that may start while the stream's previous kernel ends; each of
// these kernels waits for that one before it touches global memory.
template <typename P>
int launch(gemm_ws* h, void (*kernel)(P), int64_t blocks, int threads, size_t smem, cudaStream_t s,
           const P& params) {
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(static_cast<unsigned>(blocks), 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  if (h->pdl) {
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
  }
  cudaError_t e = cudaSuccess;
  if (smem > kDefaultSmem) e = allow_smem(h, reinterpret_cast<const void*>(kernel), smem);
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, kernel, params);
  return e == cudaSuccess ? GEMM_WS_OK : cuda_fail(h, e);
}

gws::Path pick_path(bool wide, int64_t cols, const gws::Dropout& drop) {
  if (!wide || cols % gws::GROUP != 0) return gws::ANY;
  return drop.on ? gws::DROP : gws::FAST;
}

// The threads of a row and the groups that each holds.
struct Team {
  int threads, vpt, rows;   // rows: of a block
};

// Up to 256 columns, or 1024 of many rows, a warp holds a row and a block has
// several (no barrier). Longer rows take a block. With few rows (less than two for each SM) every
// thread takes one group, for the shortest row; with many, two, and from 2048
// columns four, so that an SM has more bytes in flight for the threads that it
// can hold (8192 x 8192 bf16: 78 us with four, 86 with two); beyond 8192 columns
// always four. On the general path, whose loads take many registers, a row longer
// than a warp's 32 groups takes a block with `any_vpt` groups a thread (8192 x 8191 bf16,
// forward: 163 us with two, 232 with one; 5000 x 4095 fp32 82 and 78; backward 8192 x 8191 bf16 314
// and 249).
Team pick_team(const gemm_ws* h, int64_t rows, int64_t cols, gws::Path path, int any_vpt) {
  const int64_t groups = ceil_div(cols, gws::GROUP);
  const bool any = path == gws::ANY;
  Team t;
  if (groups <= 32 || (!any && groups <= 128 && rows >= 2 * h->num_sms)) {
    t.vpt = groups <= 32 ? 1 : groups <= 64 ? 2 : 4;
    t.threads = 32;
    t.rows = rows >= 8 * h->num_sms ? 8 : rows >= 2 * h->num_sms ? 4 : 1;
    return t;
  }
  const bool many = rows >= (any ? 8 : 2) * h->num_sms;
  t.vpt = groups > 1024 ? 4 : !many ? 1 : any ? any_vpt : groups >= 256 ? 4 : 2;
  t.threads = static_cast<int>(ceil_div(ceil_div(groups, t.vpt), 32) * 32);
  t.rows = 1;
  return t;
}

// The forward pass's `any_vpt`.
template <typename T>
constexpr int kAnyVpt = sizeof(T) == 2 ? 2 : 1;

// The ring needs some rows of each SM to be worth its set-up.
constexpr int64_t kRingRows = 4;

// How the rows pass through the ring: four groups a thread, the smallest teams
// that hold a row, and two rows at least for each team; of fp32 (8192 columns, say) two
// groups and larger teams where the ring has not that many rows (of 16-bit types it always
// has: teams * 2 rows of 3 matrices are at most 16384 * 2 * 3 * 2 bytes). *vpt: which. False
// where two rows do not fit, or a row is more than a CTA's warps hold.
template <typename Q>
bool plan_ring(int64_t cols, int64_t size, int inputs, Q* q, int* vpt) {
  const int64_t row = cols * size, groups = cols / gws::GROUP;
  int64_t room = gws::RING_BYTES / (inputs * row);
  if (room > gws::RING_MAX_STAGES) room = gws::RING_MAX_STAGES;
  for (*vpt = 4; *vpt >= (size == 2 ? 4 : 2); *vpt /= 2) {
    const int64_t warps = ceil_div(groups, 32 * *vpt);
    if (warps > gws::RING_WARPS) return false;
    q->row_bytes = static_cast<uint32_t>(row);
    q->p.team = static_cast<int>(32 * warps);
    q->teams = static_cast<int>(gws::RING_WARPS / warps);
    q->stages = static_cast<int>(room / q->teams);
    if (q->stages >= 2) return true;
  }
  return false;
}

// The kernel instance for a team and a path. Fewer threads a block leave each
// more registers: 64 with 1024, 128 with 512. NARROW: four groups a thread and at
// most 256 threads, in 16 bits kept to 80 registers, so that an SM holds three rows of
// 8192 columns (78 us; 84 with two). TWO: 2, or 1 where no team of the path has two groups
// a thread.
#define LM_NORM_INSTANCE(KERNEL, NARROW, TWO, T, PATH, ...)                         \
  (t.vpt == 1                  ? gws::KERNEL<T, PATH, 1, 1024, ##__VA_ARGS__>       \
   : t.vpt == 2                ? gws::KERNEL<T, PATH, TWO, 1024 / TWO, ##__VA_ARGS__> \
   : t.threads * t.rows <= 256 ? gws::KERNEL<T, PATH, 4, NARROW, ##__VA_ARGS__>     \
   : t.threads * t.rows <= 512 ? gws::KERNEL<T, PATH, 4, 512, ##__VA_ARGS__>        \
                               : gws::KERNEL<T, PATH, 4, 1024, ##__VA_ARGS__>)

template <typename T, int Q>
int launch_norm(gemm_ws* h, const Team& t, gws::Path path, const gws::NormParams& p, cudaStream_t s) {
  // 8 bits are for serving: with dropout they take the general path, with the aligned one's teams
  auto kernel =
      LM_NORM_INSTANCE(add_rms_norm_kernel, 512, (Q > 0 ? 2 : kAnyVpt<T>), T, gws::ANY, Q);
  if (path == gws::FAST) kernel = LM_NORM_INSTANCE(add_rms_norm_kernel, 256, 2, T, gws::FAST, Q);
  if constexpr (Q == 0)
    if (path == gws::DROP) kernel = LM_NORM_INSTANCE(add_rms_norm_kernel, 512, 2, T, gws::DROP, Q);
  return launch(h, kernel, ceil_div(p.rows, t.rows), t.threads * t.rows, 0, s, p);
}

template <typename T>
int launch_norm(gemm_ws* h, int output, const Team& t, gws::Path path, const gws::NormParams& p,
                cudaStream_t s) {
  switch (output) {
    case GEMM_WS_NORM_SAME: return launch_norm<T, 0>(h, t, path, p, s);
    case GEMM_WS_NORM_E4M3_ROW: return launch_norm<T, 1>(h, t, path, p, s);
    default: return launch_norm<T, 2>(h, t, path, p, s);
  }
}

// Elements between the blocks' rows of dweight partials: whole groups.
int64_t partial_pitch(int64_t cols) { return ceil_div(cols, gws::GROUP) * gws::GROUP; }

template <typename T>
int launch_dweight(gemm_ws* h, const float* partial, int64_t blocks, int cols, void* dweight,
                   cudaStream_t s) {
  gws::DweightParams q;
  q.partial = partial;
  q.blocks = static_cast<int>(blocks);
  q.cols = cols;
  q.pitch = static_cast<int>(partial_pitch(cols));
  q.dweight = dweight;
  return launch(h, gws::dweight_kernel<T>, ceil_div(cols, gws::DW_COLS),
                gws::DW_THREADS, 0, s, q);
}

template <typename T, bool ON>
auto ring_kernel(int vpt) {
  auto kernel = gws::add_rms_norm_grad_ring_kernel<T, ON, 4>;
  if constexpr (sizeof(T) == 4)
    if (vpt == 2) kernel = gws::add_rms_norm_grad_ring_kernel<T, ON, 2>;
  return kernel;
}

template <typename T>
int launch_grad_ring(gemm_ws* h, int vpt, const gws::NormGradRing& q, void* dweight,
                     cudaStream_t s) {
  const int64_t blocks = h->num_sms;
  const int rc = launch(h, q.p.drop.on ? ring_kernel<T, true>(vpt) : ring_kernel<T, false>(vpt),
                        blocks, gws::RING_THREADS, gws::RING_BYTES, s, q);
  if (rc != GEMM_WS_OK || !dweight) return rc;
  return launch_dweight<T>(h, q.p.partial, blocks, q.p.cols, dweight, s);
}

template <typename T>
int launch_grad(gemm_ws* h, const Team& t, gws::Path path, const gws::NormGradParams& p, void* dweight,
                cudaStream_t s) {
  const auto kernel = path == gws::ANY    ? LM_NORM_INSTANCE(add_rms_norm_grad_kernel, 512, 1, T, gws::ANY)
                      : path == gws::FAST ? LM_NORM_INSTANCE(add_rms_norm_grad_kernel, 512, 2, T, gws::FAST)
                                          : LM_NORM_INSTANCE(add_rms_norm_grad_kernel, 512, 2, T, gws::DROP);
  const int threads = t.threads * t.rows;
  const size_t smem = t.rows > 1 ? t.rows * partial_pitch(p.cols) * sizeof(float) : 0;   // at most 32 KB
  // As many blocks as run at once (1024 threads of an SM, 512 with more than one group
  // each), no more than the partials have room for.
  int64_t blocks = ceil_div(p.rows, t.rows);
  const int held = t.vpt == 1 ? 1024 : 512;
  const int64_t resident = static_cast<int64_t>(h->num_sms) * (threads >= held ? 1 : held / threads);
  if (blocks > resident) blocks = resident;
  const int64_t room = h->num_sms * kPartialPerSm / partial_pitch(p.cols);
  if (p.partial && blocks > room) blocks = room;
  const int rc = launch(h, kernel, blocks, threads, smem, s, p);
  if (rc != GEMM_WS_OK || !dweight) return rc;
  return launch_dweight<T>(h, p.partial, blocks, p.cols, dweight, s);
}

template <typename T>
int launch_dropout(gemm_ws* h, bool flat, int64_t blocks, const gws::DropoutParams& p,
                   cudaStream_t s) {
  return launch(h,
                !flat       ? gws::dropout_rows_kernel<T>
                : p.drop.on ? gws::dropout_flat_kernel<T, true>
                            : gws::dropout_flat_kernel<T, false>,
                blocks, gws::DROP_THREADS, 0, s, p);
}

}  // namespace

extern "C" {

int gemm_ws_dropout(gemm_ws_t* h, int dtype, const void* x, int64_t ldx, void* y, int64_t ldy,
                    int64_t rows, int64_t cols, double p, const uint64_t* rng, void* stream) {
  if (!h || dtype < GEMM_WS_BF16 || dtype > GEMM_WS_F32 || rows < 0 || cols < 0 ||
      rows > kMaxDim || cols > kMaxDim)
    return GEMM_WS_ERR_INVALID_ARG;
  gws::DropoutParams q;
  std::memset(&q, 0, sizeof q);
  if (!make_dropout(h, p, rng, &q.drop)) return GEMM_WS_ERR_INVALID_ARG;
  if (rows == 0 || cols == 0) return GEMM_WS_OK;
  const int64_t size = element_size(dtype);
  const Mat mx{x, ldx, size}, my{y, ldy, size};
  const Mat mr{q.drop.on ? rng : nullptr, 2, 8};
  if (!x || !y || bad_matrix(mx, cols) || bad_matrix(my, cols)) return GEMM_WS_ERR_INVALID_ARG;
  if (clash(my, mx, rows, cols, true) ||
      (mr.given() && overlaps(y, my.bytes(rows, cols), rng, 16)))
    return GEMM_WS_ERR_INVALID_ARG;
  q.x = x;
  q.y = y;
  q.ldx = ldx;
  q.ldy = ldy;
  q.rows = rows;
  q.cols = static_cast<int>(cols);
  q.groups = ceil_div(cols, gws::GROUP);
  const bool wide = mx.wide() && my.wide();
  q.row_threads = 1;
  while (q.row_threads < gws::DROP_THREADS && q.row_threads < q.groups) q.row_threads *= 2;
  const bool flat = wide && cols % gws::GROUP == 0 && (rows == 1 || (ldx == cols && ldy == cols));
  int64_t blocks = ceil_div(rows, gws::DROP_THREADS / q.row_threads);
  if (flat) {
    q.groups *= rows;
    blocks = ceil_div(q.groups, gws::DROP_THREADS * gws::DROP_VPT);
  }
  if (blocks > kMaxDim) return GEMM_WS_ERR_INVALID_ARG;
  DeviceGuard guard(h->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (dtype) {
    case GEMM_WS_BF16: return launch_dropout<__nv_bfloat16>(h, flat, blocks, q, s);
    case GEMM_WS_F16: return launch_dropout<__half>(h, flat, blocks, q, s);
    default: return launch_dropout<float>(h, flat, blocks, q, s);
  }
}

int gemm_ws_add_rms_norm(gemm_ws_t* h, int dtype, const void* x, int64_t ldx,
                         const void* residual, int64_t ldr, const void* weight, void* hidden,
                         int64_t ldh, void* y, int64_t ldy, int output, float* scales,
                         float* rstd, int64_t rows, int64_t cols, float eps, double p,
                         const uint64_t* rng, void* stream) {
  if (!h || dtype < GEMM_WS_BF16 || dtype > GEMM_WS_F32 || output < GEMM_WS_NORM_SAME ||
      output > GEMM_WS_NORM_E4M3_GROUP || rows < 0 || rows > kMaxDim || cols < 1 ||
      cols > kMaxCols || !(eps >= 0.0f))
    return GEMM_WS_ERR_INVALID_ARG;
  gws::NormParams q;
  std::memset(&q, 0, sizeof q);
  if (!make_dropout(h, p, rng, &q.drop)) return GEMM_WS_ERR_INVALID_ARG;
  if (rows == 0) return GEMM_WS_OK;
  const bool same = output == GEMM_WS_NORM_SAME;
  const int64_t size = element_size(dtype);
  const int64_t per_row = output == GEMM_WS_NORM_E4M3_GROUP ? ceil_div(cols, gws::QUANT_GROUP) : 1;
  const Mat in[3] = {{x, ldx, size}, {residual, ldr, size}, {weight, cols, size}};
  const Mat mh{hidden, ldh, size}, my{y, ldy, same ? size : 1};
  if (!x || !weight || !y || (!same && !scales)) return GEMM_WS_ERR_INVALID_ARG;
  for (const Mat& m : in)
    if (bad_matrix(m, cols)) return GEMM_WS_ERR_INVALID_ARG;
  if (bad_matrix(mh, cols) || bad_matrix(my, cols) ||
      reinterpret_cast<uintptr_t>(scales) % 4 != 0 || reinterpret_cast<uintptr_t>(rstd) % 4 != 0)
    return GEMM_WS_ERR_INVALID_ARG;
  // Outputs against the inputs and against each other.
  const Mat vec[4] = {{same ? nullptr : scales, per_row, 4}, {rstd, 1, 4}, {weight, 0, size},
                      {q.drop.on ? rng : nullptr, 0, 8}};
  const int64_t vec_bytes[4] = {rows * per_row * 4, rows * 4, cols * size, 16};
  const Mat mats[4] = {in[0], in[1], mh, my};
  if (clash(mh, in[0], rows, cols, true) || clash(mh, in[1], rows, cols, true) ||
      clash(my, in[0], rows, cols, true) || clash(my, in[1], rows, cols, false) ||
      clash(my, mh, rows, cols, false))
    return GEMM_WS_ERR_INVALID_ARG;
  for (int i = 0; i < 4; ++i)
    for (int j = 0; j < 4; ++j) {
      // scales and rstd against every matrix, weight and rng against the outputs
      if (mats[j].given() && (i < 2 || j >= 2) &&
          overlaps(vec[i].ptr, vec_bytes[i], mats[j].ptr, mats[j].bytes(rows, cols)))
        return GEMM_WS_ERR_INVALID_ARG;
      if (i < 2 && j > i && overlaps(vec[i].ptr, vec_bytes[i], vec[j].ptr, vec_bytes[j]))
        return GEMM_WS_ERR_INVALID_ARG;
    }
  q.x = x;
  q.residual = residual;
  q.weight = weight;
  q.h = hidden;
  q.y = y;
  q.rstd = rstd;
  q.scales = scales;
  q.ldx = ldx;
  q.ldr = ldr;
  q.ldh = ldh;
  q.ldy = ldy;
  q.rows = rows;
  q.cols = static_cast<int>(cols);
  q.eps = eps;
  const bool wide = in[0].wide() && (!residual || in[1].wide()) &&
           reinterpret_cast<uintptr_t>(weight) % 16 == 0 && (!hidden || mh.wide()) && my.wide();
  const gws::Path path = pick_path(wide, cols, q.drop);
  DeviceGuard guard(h->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  gws::NormRing ring;
  int vpt = 0;
  if (path == gws::DROP && same && size == 2 && rows >= kRingRows * h->num_sms) {
    ring.p = q;
    ring.status = h->work + 1;
    ring.timeout_ns = h->timeout_ns;
#ifdef GEMM_WS_DEBUG
    ring.debug_fault = h->debug_fault;
#endif
    if (plan_ring(cols, size, residual ? 2 : 1, &ring, &vpt)) {
      return launch(h,
                    dtype == GEMM_WS_BF16 ? gws::add_rms_norm_ring_kernel<__nv_bfloat16, 4>
                                          : gws::add_rms_norm_ring_kernel<__half, 4>,
                    h->num_sms, gws::RING_THREADS, gws::RING_BYTES, s, ring);
    }
  }
  const Team t = pick_team(h, rows, cols, path, size == 2 ? kAnyVpt<__half> : kAnyVpt<float>);
  q.team = t.threads;
  switch (dtype) {
    case GEMM_WS_BF16: return launch_norm<__nv_bfloat16>(h, output, t, path, q, s);
    case GEMM_WS_F16: return launch_norm<__half>(h, output, t, path, q, s);
    default: return launch_norm<float>(h, output, t, path, q, s);
  }
}

int gemm_ws_add_rms_norm_backward(gemm_ws_t* h, int dtype, const void* dy, int64_t lddy,
                                  const void* dhidden, int64_t lddh, const void* hidden,
                                  int64_t ldh, const void* weight, const float* rstd, void* dx,
                                  int64_t lddx, void* dresidual, int64_t lddr, void* dweight,
                                  int64_t rows, int64_t cols, double p, const uint64_t* rng,
                                  void* stream) {
  if (!h || dtype < GEMM_WS_BF16 || dtype > GEMM_WS_F32 || rows < 0 || rows > kMaxDim ||
      cols < 1 || cols > kMaxCols)
    return GEMM_WS_ERR_INVALID_ARG;
  gws::NormGradParams q;
  std::memset(&q, 0, sizeof q);
  if (!make_dropout(h, p, rng, &q.drop)) return GEMM_WS_ERR_INVALID_ARG;
  const int64_t size = element_size(dtype);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (reinterpret_cast<uintptr_t>(dweight) % size != 0) return GEMM_WS_ERR_INVALID_ARG;
  if (rows == 0) {
    if (!dweight) return GEMM_WS_OK;
    DeviceGuard guard(h->device);
    const cudaError_t e = cudaMemsetAsync(dweight, 0, static_cast<size_t>(cols * size), s);
    return e == cudaSuccess ? GEMM_WS_OK : cuda_fail(h, e);
  }
  const Mat in[3] = {{dy, lddy, size}, {dhidden, lddh, size}, {hidden, ldh, size}};
  const Mat out[2] = {{dx, lddx, size}, {dresidual, lddr, size}};
  if (!dy || !hidden || !weight || !rstd || !dx) return GEMM_WS_ERR_INVALID_ARG;
  for (const Mat& m : in)
    if (bad_matrix(m, cols)) return GEMM_WS_ERR_INVALID_ARG;
  for (const Mat& m : out)
    if (bad_matrix(m, cols)) return GEMM_WS_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(weight) % size != 0 || reinterpret_cast<uintptr_t>(rstd) % 4 != 0)
    return GEMM_WS_ERR_INVALID_ARG;
  const Mat vec[3] = {{weight, 0, size}, {rstd, 0, 4}, {q.drop.on ? rng : nullptr, 0, 8}};
  const int64_t vec_bytes[3] = {cols * size, rows * 4, 16};
  for (const Mat& o : out) {
    if (clash(o, in[0], rows, cols, true) || clash(o, in[1], rows, cols, true) ||
        clash(o, in[2], rows, cols, false))
      return GEMM_WS_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i)
      if (o.given() && overlaps(vec[i].ptr, vec_bytes[i], o.ptr, o.bytes(rows, cols)))
        return GEMM_WS_ERR_INVALID_ARG;
    if (o.given() && overlaps(dweight, cols * size, o.ptr, o.bytes(rows, cols)))
      return GEMM_WS_ERR_INVALID_ARG;
  }
  if (clash(out[1], out[0], rows, cols, false)) return GEMM_WS_ERR_INVALID_ARG;
  for (const Mat& m : in)
    if (m.given() && overlaps(dweight, cols * size, m.ptr, m.bytes(rows, cols)))
      return GEMM_WS_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (overlaps(dweight, cols * size, vec[i].ptr, vec_bytes[i])) return GEMM_WS_ERR_INVALID_ARG;
  q.dy = dy;
  q.dh = dhidden;
  q.h = hidden;
  q.weight = weight;
  q.rstd = rstd;
  q.dx = dx;
  q.dres = dresidual;
  q.partial = dweight ? h->partial : nullptr;
  q.lddy = lddy;
  q.lddh = lddh;
  q.ldh = ldh;
  q.lddx = lddx;
  q.lddres = lddr;
  q.rows = rows;
  q.cols = static_cast<int>(cols);
  const bool wide = in[0].wide() && (!dhidden || in[1].wide()) && in[2].wide() && out[0].wide() &&
           (!dresidual || out[1].wide()) && reinterpret_cast<uintptr_t>(weight) % 16 == 0;
  const gws::Path path = pick_path(wide, cols, q.drop);
  DeviceGuard guard(h->device);
  gws::NormGradRing ring;
  int vpt = 0;
  const Team t = pick_team(h, rows, cols, path, 1);
  // The ring from one row of each SM on, but four where the other kernel's threads hold
  // one or two groups: that starts sooner. (With dweight, bf16: 600 x 4096 8.1 us, 16.7
  // without the ring; 600 x 512 5.1 and 4.4, 200 x 4096 with one group a thread 7.2 and 5.9.)
  if (path != gws::ANY && rows >= (t.vpt == 4 ? 1 : kRingRows) * h->num_sms) {
    ring.p = q;
    ring.status = h->work + 1;
    ring.timeout_ns = h->timeout_ns;
#ifdef GEMM_WS_DEBUG
    ring.debug_fault = h->debug_fault;
#endif
    if (plan_ring(cols, size, dhidden ? 3 : 2, &ring, &vpt)) {
      switch (dtype) {
        case GEMM_WS_BF16: return launch_grad_ring<__nv_bfloat16>(h, vpt, ring, dweight, s);
        case GEMM_WS_F16: return launch_grad_ring<__half>(h, vpt, ring, dweight, s);
        default: return launch_grad_ring<float>(h, vpt, ring, dweight, s);
      }
    }
  }
  q.team = t.threads;
  switch (dtype) {
    case GEMM_WS_BF16: return launch_grad<__nv_bfloat16>(h, t, path, q, dweight, s);
    case GEMM_WS_F16: return launch_grad<__half>(h, t, path, q, dweight, s);
    default: return launch_grad<float>(h, t, path, q, dweight, s);
  }
}

#ifdef GEMM_WS_DEBUG
int gemm_ws_debug_row_columns(int64_t cols, int64_t first, int count, int* rows) {
  if (cols < 1 || cols > kMaxDim || first < 0 || first > kMaxDim / gws::GROUP + 1 || count < 0 || !rows)
    return GEMM_WS_ERR_INVALID_ARG;
  const int end = static_cast<int>(cols), groups = static_cast<int>(ceil_div(cols, gws::GROUP));
  for (int i = 0; i < count; ++i) {
    const int c = gws::column_of(static_cast<int>(first) + i, groups, end);
    int* r = rows + 3 * i;
    r[0] = c;
    r[1] = gws::has_columns(c, gws::GROUP, end);
    r[2] = gws::has_columns(c, 2 * gws::GROUP, end);
  }
  return GEMM_WS_OK;
}
#endif

}  // extern "C"
