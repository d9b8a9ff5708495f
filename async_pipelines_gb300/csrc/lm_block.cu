// Host side of the norms around a block and of the quantisation of rows
// (include/gemm_ws_lm.h): argument checks, the choice of a row's team of threads, and
// the launches.
#include <cstring>

#include "lm_host.cuh"
#include "lm_block_kernel.cuh"

static_assert(static_cast<int>(gws::Q_SAME) == GEMM_WS_NORM_SAME &&
                  static_cast<int>(gws::Q_E4M3_ROW) == GEMM_WS_NORM_E4M3_ROW &&
                  static_cast<int>(gws::Q_E4M3_GROUP) == GEMM_WS_NORM_E4M3_GROUP &&
                  static_cast<int>(gws::Q_INT8_ROW) == GEMM_WS_NORM_INT8_ROW,
              "the kernels' outputs are the interface's");

namespace {

constexpr int64_t kMaxCols = 16384;           // of a norm: its sums for each column fit shared memory
constexpr int64_t kMaxQuantCols = 32768;      // a block holds a row
// fp32 partials of the handle: two rows of kMaxCols for each SM.
constexpr int64_t kPartialPerSm = int64_t{128} * 256;
static_assert(kPartialPerSm >= 2 * kMaxCols, "a block's partial sums fit its SM's share");

// Elements between the blocks' rows of partial sums: whole groups.
int64_t partial_pitch(int64_t cols) { return ceil_div(cols, gws::GROUP) * gws::GROUP; }

// The general path's teams: a warp for short rows, up to 8 of them a block, or a block whose
// threads take one group each where rows are few, and else `most` one after the other (8192 x 8191 bf16 forward
// with four 191 us, with two 234; gradient of 2000 x 4001 104 and 82).
Team any_team(const gemm_ws* h, int64_t rows, int64_t cols, int most) {
  const int64_t groups = ceil_div(cols, gws::GROUP);
  Team t = {32, 1, 1};
  if (groups <= 32) {
    t.rows = rows >= 8 * h->num_sms ? 8 : rows >= 2 * h->num_sms ? 4 : 1;
    return t;
  }
  const int64_t threads = ceil_div(groups, rows >= 8 * h->num_sms ? most : 1);
  t.threads = static_cast<int>(threads > gws::ANY_MOST ? gws::ANY_MOST : ceil_div(threads, 32) * 32);
  return t;
}

// The rings need some rows of each SM to be worth their set-up.
constexpr int64_t kRingRows = 4;

// How the rows pass through a ring: `most` groups a thread or half as many, the smallest teams that hold
// a row, and two rows at least for each team. `vectors`: rows behind the ring. Returns the groups a
// thread; 0 where two rows do not fit, or a row is more than a CTA's warps hold.
int plan_ring(const gemm_ws* h, int64_t cols, int64_t size, int inputs, int vectors, int most, int* team,
              gws::RingPlan* q) {
  const int64_t row = cols * size, groups = cols / gws::GROUP;
  int64_t room = (gws::RING_BYTES - vectors * row) / (inputs * row);
  if (room > gws::RING_MAX_STAGES) room = gws::RING_MAX_STAGES;
  for (int vpt = most; vpt >= most / 2 && vpt > 0; vpt /= 2) {
    const int64_t warps = ceil_div(groups, 32 * vpt);
    if (warps > gws::RING_WARPS) return 0;
    std::memset(q, 0, sizeof *q);
    q->row_bytes = static_cast<uint32_t>(row);
    *team = static_cast<int>(32 * warps);
    q->teams = static_cast<int>(gws::RING_WARPS / warps);
    q->stages = static_cast<int>(room / q->teams);
    q->status = h->work + 1;
    q->timeout_ns = h->timeout_ns;
#ifdef GEMM_WS_DEBUG
    q->debug_fault = h->debug_fault;
#endif
    if (q->stages >= 2) return vpt;
  }
  return 0;
}

template <typename T, bool BYTES>
auto block_kernel(const Team& t, bool late) {
  const bool small = t.threads * t.rows <= 256;
  return t.vpt == 1   ? gws::block_norm_kernel<T, 1, 1024, BYTES, false>
         : t.vpt == 2 ? gws::block_norm_kernel<T, 2, 512, BYTES, false>
         : !late      ? gws::block_norm_kernel<T, 4, 512, BYTES, false>
         : small      ? gws::block_norm_kernel<T, 4, 256, BYTES, true>
                      : gws::block_norm_kernel<T, 4, 512, BYTES, true>;
}

template <typename T, bool BYTES>
int launch_block(gemm_ws* h, bool fast, gws::BlockParams& p, cudaStream_t s) {
  // The ring for long rows: of 16-bit types where a block's registers hold one row at a time (2000 x
  // 12000 bf16 42 us, 50 without), of fp32 from 1024 columns on (4096 x 8192 87 us and 109; 16384 x
  // 256 bf16 11 and 7).
  constexpr int MOST = sizeof(T) == 2 ? 4 : 2;
  if (fast && p.rows >= kRingRows * h->num_sms && p.cols > (sizeof(T) == 2 ? 8192 : 1023)) {
    gws::RingPlan q;
    const int vpt = plan_ring(h, p.cols, sizeof(T), p.ldg ? 3 : 2, sizeof(T) == 2 ? 3 : 0, MOST, &p.team, &q);
    auto kernel = gws::block_norm_ring_kernel<T, MOST, BYTES>;
    if constexpr (sizeof(T) == 4)
      if (vpt == 1) kernel = gws::block_norm_ring_kernel<T, 1, BYTES>;
    if (vpt)
      return launch(h, kernel, h->num_sms, gws::RING_THREADS, gws::RING_BYTES, s, p, q);
  }
  const Team t = fast ? pick_team(h, p.rows, p.cols, gws::FAST, 1) : any_team(h, p.rows, p.cols, 4);
  p.team = t.threads;
  const int64_t blocks = ceil_div(p.rows, t.rows);
  if (!fast)
    return launch_sized(h, gws::block_norm_any_kernel<T>, blocks, t.threads * t.rows,
                        t.rows * partial_pitch(p.cols) * sizeof(float), kMaxCols * sizeof(float), s, p);
  return launch(h, block_kernel<T, BYTES>(t, p.ldg == 0 && p.rows >= 8 * h->num_sms), blocks, t.threads * t.rows, 0, s, p);
}

template <typename T>
int launch_block(gemm_ws* h, bool fast, gws::BlockParams& p, cudaStream_t s) {
  return p.quant == gws::Q_SAME ? launch_block<T, false>(h, fast, p, s) : launch_block<T, true>(h, fast, p, s);
}

template <typename T>
int launch_quantize(gemm_ws* h, bool fast, gws::QuantizeParams& p, cudaStream_t s) {
  const Team t = fast ? pick_team(h, p.rows, p.cols, gws::FAST, 1) : any_team(h, p.rows, p.cols, 4);
  p.team = t.threads;
  // Four groups a thread in blocks of up to 512 threads, of which an SM then holds three (16-bit types: 4096 x 16384
  // 41 us, 48 with the registers of blocks of up to 1024).
  auto kernel = !fast                       ? gws::quantize_rows_any_kernel<T>
                : t.vpt == 1                ? gws::quantize_rows_kernel<T, 1, 1024>
                : t.vpt == 2                ? gws::quantize_rows_kernel<T, 2, 512>
                : t.threads * t.rows <= 512 ? gws::quantize_rows_kernel<T, 4, 512>
                                            : gws::quantize_rows_kernel<T, 4, 1024>;
  return launch(h, kernel, ceil_div(p.rows, t.rows), t.threads * t.rows, 0, s, p);
}

// The gradient's teams on the aligned path: a thread keeps two sums for each of its columns, so
// it takes at most two groups.
Team grad_team(const gemm_ws* h, int64_t rows, int64_t cols) {
  const int64_t groups = cols / gws::GROUP;
  Team t;
  if (groups <= 32 || (groups <= 64 && rows >= 2 * h->num_sms)) {
    t.vpt = groups <= 32 ? 1 : 2;
    t.threads = 32;
    t.rows = rows >= 8 * h->num_sms ? 8 : rows >= 2 * h->num_sms ? 4 : 1;
    return t;
  }
  t.vpt = groups > 1024 || rows >= 2 * h->num_sms ? 2 : 1;
  t.threads = static_cast<int>(ceil_div(ceil_div(groups, t.vpt), 32) * 32);
  t.rows = 1;
  return t;
}

template <typename T>
int launch_sums(gemm_ws* h, gws::BlockSumsParams& q, cudaStream_t s) {
  q.columns = static_cast<int>(ceil_div(q.cols, gws::DW_COLS));
  return launch(h, gws::block_sums_kernel<T>, int64_t{q.columns} * (q.partial && q.partial_s ? 2 : 1),
                gws::DW_THREADS, 0, s, q);
}

template <typename T>
int launch_grad(gemm_ws* h, bool fast, gws::BlockGradParams& p, gws::BlockSumsParams& q, bool first,
                bool second, cudaStream_t s) {
  const int64_t sums = first + second;
  auto finish = [&](int rc, int64_t blocks) {
    if (rc != GEMM_WS_OK || !sums) return rc;
    q.partial = p.partial;
    q.partial_s = p.partial_s;
    q.blocks = static_cast<int>(blocks);
    q.cols = p.cols;
    q.pitch = static_cast<int>(partial_pitch(p.cols));
    return launch_sums<T>(h, q, s);
  };
  auto place = [&](int64_t blocks) {
    p.partial = first ? h->partial : nullptr;
    p.partial_s = second ? h->partial + (first ? blocks * partial_pitch(p.cols) : 0) : nullptr;
  };
  // 16384 x 256 bf16 without the ring 16.4 us, with it 17.7; 16384 x 1024 49 and 47
  if (fast && p.rows >= h->num_sms && p.cols >= 1024) {
    gws::RingPlan r;
    const int vpt = plan_ring(h, p.cols, sizeof(T), 3 + (p.dh ? 1 : 0) + (p.ldg ? 1 : 0), sizeof(T) == 2 ? 3 : 0,
                              sizeof(T) == 2 ? 2 : 1, &p.team, &r);
    if (vpt) {
      place(h->num_sms);
      auto kernel = gws::block_norm_grad_ring_kernel<T, 1>;
      if constexpr (sizeof(T) == 2)
        if (vpt == 2) kernel = gws::block_norm_grad_ring_kernel<T, 2>;
      return finish(launch(h, kernel, h->num_sms, gws::RING_THREADS, gws::RING_BYTES, s, p, r), h->num_sms);
    }
  }
  Team t = fast ? grad_team(h, p.rows, p.cols) : any_team(h, p.rows, p.cols, 2);
  // Rows of which a thread would hold two groups, and the block more threads than have registers for the sums besides
  // (in 16 bits above 8192 columns: 4096 x 16384 bf16 298 us, 398 with what does not fit in local memory; fp32
  // above 4096: without the first norm 4096 x 8192 191 and 219, 8192 x 4104 241 and 271, with it 234 and 234, 296 and
  // 320; only at 8192 columns with it, a channel's gate and no dh are the registers ahead, 223 and 212).
  const bool wide = fast && t.vpt == 2 && t.threads > (sizeof(T) == 4 ? 256 : 512);
  if (wide) t.threads = 1024;
  p.team = t.threads;
  auto kernel = wide                           ? gws::block_norm_grad_any_kernel<T, true>
                : !fast                        ? gws::block_norm_grad_any_kernel<T, false>
                : t.vpt == 1                   ? gws::block_norm_grad_kernel<T, 1, 1024>
                                               : gws::block_norm_grad_kernel<T, 2, 512>;
  const int threads = t.threads * t.rows;
  const int64_t pitch = partial_pitch(p.cols);
  // at most 16 KB on the aligned path, 192 KB on the general one and of wide rows
  const size_t smem = (fast && !wide ? (t.rows > 1 ? t.rows : 0) : 3 * t.rows) * pitch * sizeof(float);
  // As many blocks as run at once, no more than the partials have room for.
  int64_t blocks = ceil_div(p.rows, t.rows);
  const int held = fast && t.vpt == 2 ? 512 : 1024;
  int64_t each = threads >= held ? 1 : held / threads;
  if (smem > 0 && each > static_cast<int64_t>(200 * 1024 / smem)) each = 200 * 1024 / smem;
  if (each < 1) each = 1;
  if (blocks > each * h->num_sms) blocks = each * h->num_sms;
  if (sums && blocks > h->num_sms * kPartialPerSm / (pitch * sums))
    blocks = h->num_sms * kPartialPerSm / (pitch * sums);
  place(blocks);
  return finish(launch_sized(h, kernel, blocks, threads, smem, 3 * kMaxCols * sizeof(float), s, p), blocks);
}

}  // namespace

extern "C" {

int gemm_ws_block_norm(gemm_ws_t* h, int dtype, const void* x, int64_t ldx, const void* residual,
                       int64_t ldr, const void* gate, int64_t ldg, const void* post_weight,
                       const void* weight, void* hidden, int64_t ldh, void* y, int64_t ldy, int output,
                       float* scales, float* post_rstd, float* rstd, int64_t rows, int64_t cols,
                       float alpha, float eps, void* stream) {
  if (!h || dtype < GEMM_WS_BF16 || dtype > GEMM_WS_F32 || output < GEMM_WS_NORM_SAME ||
      output > GEMM_WS_NORM_INT8_ROW || rows < 0 || rows > kMaxDim || cols < 1 || cols > kMaxCols ||
      !(eps >= 0.0f) || !(alpha - alpha == 0.0f))
    return GEMM_WS_ERR_INVALID_ARG;
  if (rows == 0) return GEMM_WS_OK;
  const bool same = output == GEMM_WS_NORM_SAME;
  const int64_t size = element_size(dtype);
  const bool each = gate && ldg != 0;   // a gate for each value
  const int64_t per_row = output == GEMM_WS_NORM_E4M3_GROUP ? ceil_div(cols, gws::QUANT_GROUP) : 1;
  const Mat mx{x, ldx, size}, mr{residual, ldr, size}, mg{gate, each ? ldg : cols, size},
      mp{post_weight, cols, size}, mw{weight, cols, size}, mh{hidden, ldh, size},
      my{y, ldy, same ? size : 1};
  if (!x || !residual || !weight || !y || (!same && !scales) || (post_rstd && !post_weight))
    return GEMM_WS_ERR_INVALID_ARG;
  for (const Mat* m : {&mx, &mr, &mg, &mp, &mw, &mh, &my})
    if (bad_matrix(*m, cols)) return GEMM_WS_ERR_INVALID_ARG;
  for (const float* f : {scales, post_rstd, rstd})
    if (reinterpret_cast<uintptr_t>(f) % 4 != 0) return GEMM_WS_ERR_INVALID_ARG;
  // hidden may be x or residual, and y may be x
  if (clash(mh, mx, rows, cols, true) || clash(mh, mr, rows, cols, true) ||
      clash(my, mx, rows, cols, true) || clash(my, mr, rows, cols, false))
    return GEMM_WS_ERR_INVALID_ARG;
  const Span inputs[] = {span(mg, each ? rows : 1, cols), span(mp, 1, cols), span(mw, 1, cols)};
  const Span matrices[] = {span(mx, rows, cols), span(mr, rows, cols)};
  const Span outputs[] = {span(mh, rows, cols), span(my, rows, cols), {same ? nullptr : scales, rows * per_row * 4},
                          {post_rstd, rows * 4}, {rstd, rows * 4}};
  const Span vectors[] = {outputs[2], outputs[3], outputs[4]};
  if (any_overlap(outputs, inputs) || any_overlap(vectors, matrices)) return GEMM_WS_ERR_INVALID_ARG;
  gws::BlockParams q;
  std::memset(&q, 0, sizeof q);
  q.x = x;
  q.residual = residual;
  q.gate = gate;
  q.post = post_weight;
  q.weight = weight;
  q.h = hidden;
  q.y = y;
  q.post_rstd = post_rstd;
  q.rstd = rstd;
  q.scales = scales;
  q.ldx = ldx;
  q.ldr = ldr;
  q.ldg = each ? ldg : 0;
  q.ldh = ldh;
  q.ldy = ldy;
  q.rows = rows;
  q.cols = static_cast<int>(cols);
  q.quant = output;
  q.alpha = alpha;
  q.eps = eps;
  const bool wide = mx.wide() && mr.wide() && (!gate || (each ? mg.wide() : aligned16(gate))) &&
                    aligned16(post_weight) && aligned16(weight) && (!hidden || mh.wide()) && my.wide();
  const bool fast = wide && cols % gws::GROUP == 0;
  DeviceGuard guard(h->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (dtype) {
    case GEMM_WS_BF16: return launch_block<__nv_bfloat16>(h, fast, q, s);
    case GEMM_WS_F16: return launch_block<__half>(h, fast, q, s);
    default: return launch_block<float>(h, fast, q, s);
  }
}

int gemm_ws_block_norm_backward(gemm_ws_t* h, int dtype, const void* dy, int64_t lddy,
                                const void* dhidden, int64_t lddh, const void* x, int64_t ldx,
                                const void* hidden, int64_t ldh, const void* gate, int64_t ldg,
                                const void* post_weight, const void* weight, const float* post_rstd,
                                const float* rstd, void* dx, int64_t lddx, void* dresidual,
                                int64_t lddr, void* dgate, int64_t lddg, void* dpost_weight,
                                void* dweight, int64_t rows, int64_t cols, float alpha, void* stream) {
  if (!h || dtype < GEMM_WS_BF16 || dtype > GEMM_WS_F32 || rows < 0 || rows > kMaxDim || cols < 1 ||
      cols > kMaxCols || !(alpha - alpha == 0.0f))
    return GEMM_WS_ERR_INVALID_ARG;
  const int64_t size = element_size(dtype);
  const bool each = gate && ldg != 0;   // a gate for each value
  if ((dgate && !gate) || (dpost_weight && !post_weight)) return GEMM_WS_ERR_INVALID_ARG;
  const Mat my{dy, lddy, size}, md{dhidden, lddh, size}, mx{x, ldx, size}, mh{hidden, ldh, size},
      mg{gate, each ? ldg : cols, size}, mp{post_weight, cols, size}, mw{weight, cols, size},
      ox{dx, lddx, size}, orr{dresidual, lddr, size}, og{dgate, each ? lddg : cols, size},
      op{dpost_weight, cols, size}, ow{dweight, cols, size};
  for (const Mat* m : {&mg, &mp, &mw, &og, &op, &ow})
    if (bad_matrix(*m, cols)) return GEMM_WS_ERR_INVALID_ARG;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (rows == 0) {
    DeviceGuard guard(h->device);
    for (void* v : {dweight, dpost_weight, each ? nullptr : dgate}) {
      if (!v) continue;
      const cudaError_t e = cudaMemsetAsync(v, 0, static_cast<size_t>(cols * size), s);
      if (e != cudaSuccess) return cuda_fail(h, e);
    }
    return GEMM_WS_OK;
  }
  if (!dy || !x || !hidden || !weight || !rstd || !dx || (post_weight && !post_rstd))
    return GEMM_WS_ERR_INVALID_ARG;
  for (const Mat* m : {&my, &md, &mx, &mh, &ox, &orr})
    if (bad_matrix(*m, cols)) return GEMM_WS_ERR_INVALID_ARG;
  for (const float* f : {post_rstd, rstd})
    if (reinterpret_cast<uintptr_t>(f) % 4 != 0) return GEMM_WS_ERR_INVALID_ARG;
  // dx and dresidual may each be dy or dhidden
  for (const Mat* o : {&ox, &orr})
    if (clash(*o, my, rows, cols, true) || clash(*o, md, rows, cols, true)) return GEMM_WS_ERR_INVALID_ARG;
  const Span inputs[] = {span(mx, rows, cols), span(mh, rows, cols), span(mg, each ? rows : 1, cols),
                         span(mp, 1, cols), span(mw, 1, cols), {post_weight ? post_rstd : nullptr, rows * 4},
                         {rstd, rows * 4}};
  const Span given[] = {span(my, rows, cols), span(md, rows, cols)};
  const Span outputs[] = {span(ox, rows, cols), span(orr, rows, cols), span(og, each ? rows : 1, cols),
                          span(op, 1, cols), span(ow, 1, cols)};
  const Span others[] = {outputs[2], outputs[3], outputs[4]};
  if (any_overlap(outputs, inputs) || any_overlap(others, given)) return GEMM_WS_ERR_INVALID_ARG;
  gws::BlockGradParams q;
  gws::BlockSumsParams sums;
  std::memset(&q, 0, sizeof q);
  std::memset(&sums, 0, sizeof sums);
  q.dy = dy;
  q.dh = dhidden;
  q.x = x;
  q.h = hidden;
  q.gate = gate;
  q.post = post_weight;
  q.weight = weight;
  q.post_rstd = post_rstd;
  q.rstd = rstd;
  q.dx = dx;
  q.dres = dresidual;
  q.dgate = each ? dgate : nullptr;
  q.lddy = lddy;
  q.lddh = lddh;
  q.ldx = ldx;
  q.ldh = ldh;
  q.ldg = each ? ldg : 0;
  q.lddx = lddx;
  q.lddres = lddr;
  q.lddg = lddg;
  q.rows = rows;
  q.cols = static_cast<int>(cols);
  q.alpha = alpha;
  sums.gate = each ? nullptr : gate;
  sums.post = post_weight;
  sums.dweight = dweight;
  sums.dpost = dpost_weight;
  sums.dgate = each ? nullptr : dgate;
  const bool wide = my.wide() && (!dhidden || md.wide()) && mx.wide() && mh.wide() &&
                    (!gate || (each ? mg.wide() : aligned16(gate))) && aligned16(post_weight) &&
                    aligned16(weight) && ox.wide() && (!dresidual || orr.wide()) &&
                    (!q.dgate || og.wide());
  const bool fast = wide && cols % gws::GROUP == 0;
  const bool second = sums.dpost || sums.dgate;
  DeviceGuard guard(h->device);
  switch (dtype) {
    case GEMM_WS_BF16: return launch_grad<__nv_bfloat16>(h, fast, q, sums, dweight, second, s);
    case GEMM_WS_F16: return launch_grad<__half>(h, fast, q, sums, dweight, second, s);
    default: return launch_grad<float>(h, fast, q, sums, dweight, second, s);
  }
}

int gemm_ws_quantize_rows(gemm_ws_t* h, int dtype, const void* x, int64_t ldx, int8_t* y, int64_t ldy,
                          float* scales, int64_t rows, int64_t cols, void* stream) {
  if (!h || dtype < GEMM_WS_BF16 || dtype > GEMM_WS_F32 || rows < 0 || rows > kMaxDim || cols < 1 ||
      cols > kMaxQuantCols)
    return GEMM_WS_ERR_INVALID_ARG;
  if (rows == 0) return GEMM_WS_OK;
  const Mat mx{x, ldx, element_size(dtype)}, my{y, ldy, 1};
  if (!x || !y || !scales || bad_matrix(mx, cols) || bad_matrix(my, cols) ||
      reinterpret_cast<uintptr_t>(scales) % 4 != 0)
    return GEMM_WS_ERR_INVALID_ARG;
  const Span inputs[] = {span(mx, rows, cols)}, outputs[] = {span(my, rows, cols), {scales, rows * 4}};
  if (any_overlap(outputs, inputs)) return GEMM_WS_ERR_INVALID_ARG;
  gws::QuantizeParams q;
  std::memset(&q, 0, sizeof q);
  q.x = x;
  q.y = y;
  q.scales = scales;
  q.ldx = ldx;
  q.ldy = ldy;
  q.rows = rows;
  q.cols = static_cast<int>(cols);
  const bool fast = mx.wide() && my.wide() && cols % gws::GROUP == 0;
  DeviceGuard guard(h->device);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  switch (dtype) {
    case GEMM_WS_BF16: return launch_quantize<__nv_bfloat16>(h, fast, q, s);
    case GEMM_WS_F16: return launch_quantize<__half>(h, fast, q, s);
    default: return launch_quantize<float>(h, fast, q, s);
  }
}

}  // extern "C"
