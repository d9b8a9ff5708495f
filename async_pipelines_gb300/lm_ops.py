"""Tensor API of the language-model operators in include/gemm_ws_lm.h.

`LmOps` holds their methods; `gemm_ws.GemmWS` inherits them, so one handle
runs the matrix products and what surrounds them. As there, outputs are the
caller's tensors, calls run asynchronously on the current (or the given)
stream, and there is no fallback.
"""
from __future__ import annotations

import ctypes

import torch

BF16, F16, F32 = 0, 1, 2                                  # gemm_ws_dtype
NORM_SAME, NORM_E4M3_ROW, NORM_E4M3_GROUP, NORM_INT8_ROW = 0, 1, 2, 3   # gemm_ws_norm_output
QUANT_GROUP = 128                                         # columns of one scale

EXPORTS = ("gemm_ws_dropout", "gemm_ws_add_rms_norm", "gemm_ws_add_rms_norm_backward",
           "gemm_ws_linear_ce", "gemm_ws_linear_ce_backward", "gemm_ws_linear_ce_workspace",
           "gemm_ws_block_norm", "gemm_ws_block_norm_backward", "gemm_ws_quantize_rows",
           "gemm_ws_int8_matmul", "gemm_ws_int8_matmul_workspace", "gemm_ws_adjust_logits")

TOKEN_BYTES = {torch.int64: 8, torch.int32: 4}
TARGET_BYTES = TOKEN_BYTES

_DTYPES = {torch.bfloat16: BF16, torch.float16: F16, torch.float32: F32}


def declare(lib) -> None:
    """Argument and result types of the entry points, on a loaded library."""
    vp, i64, f32, f64, i32 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_float, ctypes.c_double,
                              ctypes.c_int)
    lib.gemm_ws_dropout.argtypes = [vp, i32, vp, i64, vp, i64, i64, i64, f64, vp, vp]
    lib.gemm_ws_add_rms_norm.argtypes = [vp, i32, vp, i64, vp, i64, vp, vp, i64, vp, i64, i32, vp,
                                         vp, i64, i64, f32, f64, vp, vp]
    lib.gemm_ws_add_rms_norm_backward.argtypes = [vp, i32, vp, i64, vp, i64, vp, i64, vp, vp, vp,
                                                  i64, vp, i64, vp, i64, i64, f64, vp, vp]
    lib.gemm_ws_linear_ce.argtypes = [vp, vp, i64, vp, i64, vp, i32, i64, vp, vp, vp, i64, i64,
                                      i64, vp, i64, vp]
    lib.gemm_ws_linear_ce_backward.argtypes = [vp, vp, i64, vp, i64, vp, i32, i64, vp, vp, i32, vp,
                                               i64, vp, i64, i64, i64, i64, vp, i64, vp]
    lib.gemm_ws_linear_ce_workspace.argtypes = [vp, i64, i64, i64, i32]
    lib.gemm_ws_block_norm.argtypes = [vp, i32, vp, i64, vp, i64, vp, i64, vp, vp, vp, i64, vp, i64,
                                       i32, vp, vp, vp, i64, i64, f32, f32, vp]
    lib.gemm_ws_block_norm_backward.argtypes = [vp, i32, vp, i64, vp, i64, vp, i64, vp, i64, vp, i64,
                                                vp, vp, vp, vp, vp, i64, vp, i64, vp, i64, vp, vp, i64,
                                                i64, f32, vp]
    lib.gemm_ws_quantize_rows.argtypes = [vp, i32, vp, i64, vp, i64, vp, i64, i64, vp]
    lib.gemm_ws_int8_matmul.argtypes = [vp, vp, i64, vp, vp, i64, vp, vp, vp, i64, i32, i64, i64, i64,
                                        vp, i64, vp]
    lib.gemm_ws_int8_matmul_workspace.argtypes = [vp, i64, i64, i64]
    lib.gemm_ws_adjust_logits.argtypes = [vp, i32, vp, i64, i32, vp, i64, vp, i32, i64, i64, vp, vp, vp,
                                          vp, vp, vp, i32, i64, vp, i64, i64, vp, i64, i64, i64, vp]
    for name in EXPORTS:
        getattr(lib, name).restype = i32
    lib.gemm_ws_linear_ce_workspace.restype = i64
    lib.gemm_ws_int8_matmul_workspace.restype = i64


def _rows(name, t, shape, dtype):
    """(pointer, elements between rows) of a matrix argument; (None, 0) for None."""
    if t is None:
        return None, 0
    if t.dtype is not dtype or not t.is_cuda or t.shape != shape:
        raise ValueError(f"{name} must be a {tuple(shape)} {dtype} CUDA tensor, got "
                         f"{tuple(t.shape)} {t.dtype} on {t.device}")
    step, inner = t.stride()
    cols = shape[1]
    if inner != 1 or step < cols:   # of one column, or one row, a stride says nothing
        if (inner != 1 and cols > 1) or (step < cols and shape[0] > 1):
            raise ValueError(f"{name} must have contiguous rows that do not overlap")
        step = max(step, cols)
    return t.data_ptr(), step


def _flat(name, t, n, dtype):
    """The pointer of a contiguous argument of n elements; None for None."""
    if t is None:
        return None
    if t.dtype is not dtype or not t.is_cuda or t.numel() != n or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of {n} elements")
    return t.data_ptr()


def _mask(p, rng):
    """The pointer of the generator's words; None where nothing is dropped."""
    if p == 0.0:
        return None
    if not 0.0 <= p <= 1.0:
        raise ValueError("p must be in [0, 1]")
    if rng is None:
        raise ValueError("dropout needs rng: an int64 CUDA tensor (seed, first counter)")
    return _flat("rng", rng, 2, torch.int64)


def _type_of(x):
    code = _DTYPES.get(x.dtype)
    if code is None or x.dim() != 2:
        raise ValueError("x must be a 2-D bf16, f16 or f32 tensor (rows, cols)")
    return code


# torch.cuda.current_stream() builds an object, which takes as long as a launch.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


class LmOps:
    """The operators' methods, on an object with `lib`, `handle` and `device`."""

    def _stream_of(self, stream) -> int:
        """The raw cudaStream_t of `stream` (default: the device's current torch stream)."""
        if stream is None:
            if _raw_stream is not None:
                return _raw_stream(self.device)
            return torch.cuda.current_stream(self.device).cuda_stream
        if isinstance(stream, torch.cuda.Stream):
            return stream.cuda_stream
        return int(stream)

    def dropout(self, x, y, p, rng, stream=None):
        """y = keep * x / (1 - p); x, y: (rows, cols) of one type; y may be x.

        rng: int64 (seed, first counter) on the GPU. The call uses
        rows * ceil(cols / 8) counters; the same words give the same mask, which
        is how the gradient is taken.
        """
        code = _type_of(x)
        px, ldx = _rows("x", x, x.shape, x.dtype)
        py, ldy = _rows("y", y, x.shape, x.dtype)
        rows, cols = x.shape
        rc = self.lib.gemm_ws_dropout(self.handle, code, px, ldx, py, ldy, rows, cols, p,
                                      _mask(p, rng), self._stream_of(stream))
        if rc:
            self._raise(rc, "gemm_ws_dropout")
        return y

    def add_rms_norm(self, x, weight, y, residual=None, h=None, rstd=None, scales=None, eps=1e-6,
                     p=0.0, rng=None, stream=None):
        """h = residual + dropout(x); y = weight * h / sqrt(mean(h^2) + eps).

        x, residual, h, y: (rows, cols); weight: (cols,). With y of type
        torch.float8_e4m3fn, scales is f32 and says how y is scaled: rows
        elements, one a row, or (rows, ceil(cols / 128)), one for each 128
        columns; y * scale is the norm. rstd: (rows,) f32, for the backward
        pass. h may be x or residual, y may be x.
        """
        code = _type_of(x)
        shape, dtype = x.shape, x.dtype
        rows, cols = shape
        px, ldx = _rows("x", x, shape, dtype)
        pr, ldr = _rows("residual", residual, shape, dtype)
        ph, ldh = _rows("h", h, shape, dtype)
        output = NORM_SAME
        ps = None
        if scales is not None:
            groups = (cols + QUANT_GROUP - 1) // QUANT_GROUP
            by_group = groups > 1 and scales.dim() == 2 and scales.shape[1] == groups
            output = NORM_E4M3_GROUP if by_group else NORM_E4M3_ROW
            ps = _flat("scales", scales, rows * groups if by_group else rows, torch.float32)
            py, ldy = _rows("y", y, shape, torch.float8_e4m3fn)
        else:
            py, ldy = _rows("y", y, shape, dtype)
        rc = self.lib.gemm_ws_add_rms_norm(
            self.handle, code, px, ldx, pr, ldr, _flat("weight", weight, cols, dtype), ph, ldh,
            py, ldy, output, ps, _flat("rstd", rstd, rows, torch.float32), rows, cols, eps, p,
            _mask(p, rng), self._stream_of(stream))
        if rc:
            self._raise(rc, "gemm_ws_add_rms_norm")
        return y

    def add_rms_norm_backward(self, dy, h, weight, rstd, dx, dweight=None, dh=None,
                              dresidual=None, p=0.0, rng=None, stream=None):
        """Gradients of add_rms_norm: dx of x, dresidual of residual, dweight.

        dy: of y; dh: what reaches h from its other uses (None: zero); h, rstd:
        what the forward call wrote; p, rng: as given to it. Without dropout
        dx is the residual's gradient too.
        """
        code = _type_of(dy)
        shape, dtype = dy.shape, dy.dtype
        rows, cols = shape
        pdy, lddy = _rows("dy", dy, shape, dtype)
        pdh, lddh = _rows("dh", dh, shape, dtype)
        ph, ldh = _rows("h", h, shape, dtype)
        pdx, lddx = _rows("dx", dx, shape, dtype)
        pdr, lddr = _rows("dresidual", dresidual, shape, dtype)
        rc = self.lib.gemm_ws_add_rms_norm_backward(
            self.handle, code, pdy, lddy, pdh, lddh, ph, ldh,
            _flat("weight", weight, cols, dtype), _flat("rstd", rstd, rows, torch.float32), pdx,
            lddx, pdr, lddr, _flat("dweight", dweight, cols, dtype), rows, cols, p,
            _mask(p, rng), self._stream_of(stream))
        if rc:
            self._raise(rc, "gemm_ws_add_rms_norm_backward")
        return dx

    # -------------------------------------------------------------- cross entropy

    def linear_cross_entropy_workspace(self, tokens, hidden, vocab, backward=False) -> int:
        """Bytes of workspace that one call needs."""
        sizes = (tokens, hidden, vocab, bool(backward))
        n = self._ce_need.get(sizes)
        if n is not None:
            return n
        n = self.lib.gemm_ws_linear_ce_workspace(self.handle, tokens, hidden, vocab,
                                                 int(bool(backward)))
        if n < 0:
            self._raise(-n, "gemm_ws_linear_ce_workspace")
        if len(self._ce_need) >= 1024:
            self._ce_need.clear()
        self._ce_need[sizes] = n
        return n

    def _workspace(self, workspace, need, x, stream):
        """(tensor, pointer, bytes): the caller's, or one from torch's allocator for this call."""
        if workspace is None:
            if stream is None:
                workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
            else:   # allocated for the stream that the call runs on
                if not isinstance(stream, torch.cuda.Stream):
                    stream = torch.cuda.ExternalStream(int(stream), device=x.device)
                with torch.cuda.stream(stream):
                    workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
        elif workspace.dtype is not torch.uint8 or not workspace.is_cuda or \
                not workspace.is_contiguous():
            raise ValueError("workspace must be a contiguous uint8 CUDA tensor")
        return workspace, workspace.data_ptr(), workspace.numel()

    def _ce_operands(self, x, weight, targets):
        bf16 = torch.bfloat16
        if x.dim() != 2 or weight.dim() != 2 or weight.shape[1] != x.shape[1]:
            raise ValueError("x must be (tokens, hidden) and weight (vocab, hidden)")
        px, ldx = _rows("x", x, x.shape, bf16)
        pw, ldw = _rows("weight", weight, weight.shape, bf16)
        size = TARGET_BYTES.get(targets.dtype)
        if size is None:
            raise ValueError("targets must be int64 or int32")
        return px, ldx, pw, ldw, _flat("targets", targets, x.shape[0], targets.dtype), size

    def linear_cross_entropy(self, x, weight, targets, loss, lse, mean=None, ignore_index=-100,
                             workspace=None, stream=None):
        """Softmax cross entropy of x @ weight^T, the logits never held.

        x: (tokens, hidden), weight: (vocab, hidden), bf16; targets: (tokens,)
        int64 or int32. loss, lse: (tokens,) f32; mean: 2 f32, the mean loss
        over the counted tokens and 1 / their number. A token whose target is
        ignore_index is not counted: loss and lse 0, its row plays no part; one
        whose target is outside the vocabulary has loss NaN. Without a
        workspace (uint8, linear_cross_entropy_workspace bytes) the call takes
        one from torch's allocator.
        """
        px, ldx, pw, ldw, pt, size = self._ce_operands(x, weight, targets)
        tokens, hidden = x.shape
        vocab = weight.shape[0]
        f32 = torch.float32
        ploss, plse = _flat("loss", loss, tokens, f32), _flat("lse", lse, tokens, f32)
        pmean = _flat("mean", mean, 2, f32)
        need = self.linear_cross_entropy_workspace(tokens, hidden, vocab)
        workspace, pws, bytes_ = self._workspace(workspace, need, x, stream)
        rc = self.lib.gemm_ws_linear_ce(
            self.handle, px, ldx, pw, ldw, pt, size, ignore_index, ploss, plse, pmean, tokens,
            hidden, vocab, pws, bytes_, self._stream_of(stream))
        if rc:
            self._raise(rc, "gemm_ws_linear_ce")
        return loss

    def linear_cross_entropy_backward(self, x, weight, targets, lse, grad, dx=None, dweight=None,
                                      ignore_index=-100, workspace=None, stream=None):
        """Gradients of sum(grad * loss): dx (tokens, hidden), dweight (vocab, hidden), bf16.

        lse: what linear_cross_entropy wrote. grad: f32, one for each token, or
        one element for all: mean[1:] gives the gradient of the mean.
        """
        px, ldx, pw, ldw, pt, size = self._ce_operands(x, weight, targets)
        tokens, hidden = x.shape
        vocab = weight.shape[0]
        bf16, f32 = torch.bfloat16, torch.float32
        step = 0 if grad.numel() == 1 else 1
        plse, pgrad = _flat("lse", lse, tokens, f32), _flat("grad", grad, tokens if step else 1, f32)
        pdx, lddx = _rows("dx", dx, x.shape, bf16)
        pdw, lddw = _rows("dweight", dweight, weight.shape, bf16)
        need = self.linear_cross_entropy_workspace(tokens, hidden, vocab, backward=True)
        workspace, pws, bytes_ = self._workspace(workspace, need, x, stream)
        rc = self.lib.gemm_ws_linear_ce_backward(
            self.handle, px, ldx, pw, ldw, pt, size, ignore_index, plse, pgrad, step, pdx, lddx,
            pdw, lddw, tokens, hidden, vocab, pws, bytes_, self._stream_of(stream))
        if rc:
            self._raise(rc, "gemm_ws_linear_ce_backward")
        return dx, dweight

    # -------------------------------------------------------------- norms around a block

    def _gate(self, name, gate, shape, dtype):
        """(pointer, elements between rows): of each channel's gate 0 elements."""
        if gate is None:
            return None, 0
        if gate.dim() == 1:
            return _flat(name, gate, shape[1], dtype), 0
        return _rows(name, gate, shape, dtype)

    def block_norm(self, x, residual, weight, y, post_weight=None, gate=None, alpha=1.0, h=None,
                   post_rstd=None, rstd=None, scales=None, eps=1e-6, stream=None):
        """h = alpha * residual + gate * post_norm(x); y = weight * h / sqrt(mean(h^2) + eps).

        post_norm(x) = post_weight * x / sqrt(mean(x^2) + eps), or x without
        post_weight. x (a block's output), residual, h, y: (rows, cols); weight,
        post_weight: (cols,); gate: (cols,), (rows, cols), or None. With y of type
        torch.int8, scales is f32 with an element for each row; with
        torch.float8_e4m3fn it is as in add_rms_norm. post_rstd, rstd: (rows,) f32,
        for the backward pass. h may be x or residual, y may be x.
        """
        code = _type_of(x)
        shape, dtype = x.shape, x.dtype
        rows, cols = shape
        px, ldx = _rows("x", x, shape, dtype)
        if residual is None:
            raise ValueError("residual must be given")
        pr, ldr = _rows("residual", residual, shape, dtype)
        pg, ldg = self._gate("gate", gate, shape, dtype)
        ph, ldh = _rows("h", h, shape, dtype)
        output = NORM_SAME
        ps = None
        if scales is None:
            py, ldy = _rows("y", y, shape, dtype)
        elif y.dtype is torch.int8:
            output = NORM_INT8_ROW
            ps = _flat("scales", scales, rows, torch.float32)
            py, ldy = _rows("y", y, shape, torch.int8)
        else:
            groups = (cols + QUANT_GROUP - 1) // QUANT_GROUP
            by_group = groups > 1 and scales.dim() == 2 and scales.shape[1] == groups
            output = NORM_E4M3_GROUP if by_group else NORM_E4M3_ROW
            ps = _flat("scales", scales, rows * groups if by_group else rows, torch.float32)
            py, ldy = _rows("y", y, shape, torch.float8_e4m3fn)
        rc = self.lib.gemm_ws_block_norm(
            self.handle, code, px, ldx, pr, ldr, pg, ldg,
            _flat("post_weight", post_weight, cols, dtype), _flat("weight", weight, cols, dtype), ph,
            ldh, py, ldy, output, ps, _flat("post_rstd", post_rstd, rows, torch.float32),
            _flat("rstd", rstd, rows, torch.float32), rows, cols, alpha, eps, self._stream_of(stream))
        if rc:
            self._raise(rc, "gemm_ws_block_norm")
        return y

    def block_norm_backward(self, dy, x, h, weight, rstd, dx, dresidual=None, post_weight=None,
                            post_rstd=None, gate=None, alpha=1.0, dh=None, dweight=None,
                            dpost_weight=None, dgate=None, stream=None):
        """Gradients of block_norm: dx, dresidual, dweight, dpost_weight and dgate.

        dy: of y; dh: what reaches h from its other uses (None: zero); x, weight,
        post_weight, gate, alpha: as given to it; h, rstd, post_rstd: what it wrote. dgate
        has the gate's shape. dx and dresidual may each be dy or dh.
        """
        code = _type_of(dy)
        shape, dtype = dy.shape, dy.dtype
        rows, cols = shape
        f32 = torch.float32
        pdy, lddy = _rows("dy", dy, shape, dtype)
        pdh, lddh = _rows("dh", dh, shape, dtype)
        px, ldx = _rows("x", x, shape, dtype)
        ph, ldh = _rows("h", h, shape, dtype)
        pg, ldg = self._gate("gate", gate, shape, dtype)
        pdx, lddx = _rows("dx", dx, shape, dtype)
        pdr, lddr = _rows("dresidual", dresidual, shape, dtype)
        if dgate is not None and (gate is None or dgate.dim() != gate.dim()):
            raise ValueError("dgate must have the gate's shape")
        pdg, lddg = self._gate("dgate", dgate, shape, dtype)
        rc = self.lib.gemm_ws_block_norm_backward(
            self.handle, code, pdy, lddy, pdh, lddh, px, ldx, ph, ldh, pg, ldg,
            _flat("post_weight", post_weight, cols, dtype), _flat("weight", weight, cols, dtype),
            _flat("post_rstd", post_rstd, rows, f32), _flat("rstd", rstd, rows, f32), pdx, lddx, pdr,
            lddr, pdg, lddg, _flat("dpost_weight", dpost_weight, cols, dtype),
            _flat("dweight", dweight, cols, dtype), rows, cols, alpha, self._stream_of(stream))
        if rc:
            self._raise(rc, "gemm_ws_block_norm_backward")
        return dx

    # -------------------------------------------------------------- 8-bit integers

    def quantize_rows(self, x, y, scales, stream=None):
        """y = x / scales in 8-bit integers, scales = max |x| / 127 of each row.

        x: (rows, cols) bf16, f16 or f32; y: (rows, cols) int8; scales: (rows,) f32.
        """
        code = _type_of(x)
        px, ldx = _rows("x", x, x.shape, x.dtype)
        py, ldy = _rows("y", y, x.shape, torch.int8)
        rows, cols = x.shape
        rc = self.lib.gemm_ws_quantize_rows(self.handle, code, px, ldx, py, ldy,
                                            _flat("scales", scales, rows, torch.float32), rows, cols,
                                            self._stream_of(stream))
        if rc:
            self._raise(rc, "gemm_ws_quantize_rows")
        return y

    def int8_matmul_workspace(self, tokens, channels, k) -> int:
        """Bytes of workspace that one call needs."""
        sizes = (tokens, channels, k)
        n = self._int8_need.get(sizes)
        if n is not None:
            return n
        n = self.lib.gemm_ws_int8_matmul_workspace(self.handle, tokens, channels, k)
        if n < 0:
            self._raise(-n, "gemm_ws_int8_matmul_workspace")
        if len(self._int8_need) >= 1024:
            self._int8_need.clear()
        self._int8_need[sizes] = n
        return n

    def int8_matmul(self, a, w, a_scales, w_scales, d, bias=None, workspace=None, stream=None):
        """d = (a @ w^T) * a_scales[:, None] * w_scales + bias, the sums exact.

        a: (tokens, k), w: (channels, k), int8, w's rows on 16-byte boundaries; a_scales:
        (tokens,), w_scales, bias: (channels,), f32; d: (tokens, channels) bf16, f16 or f32.
        Without a workspace (uint8, int8_matmul_workspace bytes) the call takes one from
        torch's allocator where it needs one.
        """
        if a.dim() != 2 or w.dim() != 2 or w.shape[1] != a.shape[1]:
            raise ValueError("a must be (tokens, k) and w (channels, k)")
        tokens, k = a.shape
        channels = w.shape[0]
        pa, lda = _rows("a", a, a.shape, torch.int8)
        pw, ldw = _rows("w", w, w.shape, torch.int8)
        code = _type_of(d)
        pd, ldd = _rows("d", d, (tokens, channels), d.dtype)
        f32 = torch.float32
        need = self.int8_matmul_workspace(tokens, channels, k)
        pws, bytes_ = None, 0
        if need > 0 or workspace is not None:
            workspace, pws, bytes_ = self._workspace(workspace, need, a, stream)
        rc = self.lib.gemm_ws_int8_matmul(
            self.handle, pa, lda, _flat("a_scales", a_scales, tokens, f32), pw, ldw,
            _flat("w_scales", w_scales, channels, f32), _flat("bias", bias, channels, f32), pd, ldd, code,
            tokens, channels, k, pws, bytes_, self._stream_of(stream))
        if rc:
            self._raise(rc, "gemm_ws_int8_matmul")
        return d

    # -------------------------------------------------------------- logits

    def adjust_logits(self, logits, out, tokens=None, lengths=None, prompt_lengths=None,
                      repetition=None, frequency=None, presence=None, bias_tokens=None,
                      bias_values=None, allowed=None, stream=None):
        """Penalties for repeated tokens, biases and masks; logits, out: (rows, vocab).

        out has the logits' type or f32, and may be the logits. tokens: (rows, history) int64
        or int32, the history, of which lengths (rows,) int32 count (None: all) and the first
        prompt_lengths (rows,) int32 are the prompt (None: nothing is). repetition divides or
        multiplies the logits of all tokens in it; frequency is taken off for each time that a
        token was generated and presence once: (rows,) f32. bias_tokens (int64 or int32) and
        bias_values (f32): (rows, n). allowed: (rows, ceil(vocab / 32)) int32, bit v % 32 of word
        v // 32 for token v; what is not allowed becomes -inf.
        """
        code = _type_of(logits)
        shape = logits.shape
        rows, vocab = shape
        f32, i32 = torch.float32, torch.int32
        if out.dtype is not logits.dtype and out.dtype is not f32:
            raise ValueError("out must have the logits' type or f32")
        pl, ldl = _rows("logits", logits, shape, logits.dtype)
        po, ldo = _rows("out", out, shape, out.dtype)
        pt, ldt, size, history = None, 0, 8, 0
        if tokens is not None:
            size = TOKEN_BYTES.get(tokens.dtype)
            if size is None or tokens.dim() != 2 or tokens.shape[0] != rows:
                raise ValueError("tokens must be (rows, history) int64 or int32")
            pt, ldt = _rows("tokens", tokens, tokens.shape, tokens.dtype)
            history = tokens.shape[1]
        elif any(v is not None for v in (lengths, prompt_lengths, repetition, frequency, presence)):
            raise ValueError("penalties need tokens")
        pb, ldb, pv, ldv, bsize, biases = None, 0, None, 0, 8, 0
        if (bias_tokens is None) != (bias_values is None):
            raise ValueError("bias_tokens and bias_values are given together")
        if bias_tokens is not None:
            bsize = TOKEN_BYTES.get(bias_tokens.dtype)
            if bsize is None or bias_tokens.dim() != 2 or bias_tokens.shape[0] != rows:
                raise ValueError("bias_tokens must be (rows, n) int64 or int32")
            pb, ldb = _rows("bias_tokens", bias_tokens, bias_tokens.shape, bias_tokens.dtype)
            pv, ldv = _rows("bias_values", bias_values, bias_tokens.shape, f32)
            biases = bias_tokens.shape[1]
        pa, lda = None, 0
        if allowed is not None:
            pa, lda = _rows("allowed", allowed, (rows, (vocab + 31) // 32), i32)
        rc = self.lib.gemm_ws_adjust_logits(
            self.handle, code, pl, ldl, _DTYPES[out.dtype], po, ldo, pt, size, ldt, history,
            _flat("lengths", lengths, rows, i32), _flat("prompt_lengths", prompt_lengths, rows, i32),
            _flat("repetition", repetition, rows, f32), _flat("frequency", frequency, rows, f32),
            _flat("presence", presence, rows, f32), pb, bsize, ldb, pv, ldv, biases, pa, lda, rows,
            vocab, self._stream_of(stream))
        if rc:
            self._raise(rc, "gemm_ws_adjust_logits")
        return out
