"""Cases of the operators around a block and of serving in 8-bit integers: what they are given, what they return, and their plain forms.

Four operators that lie between a block's output and the next token, as methods of `gemm_ws.GemmWS`:

* block_norm      the norm after a block, its gate, the scaled residual and the norm before the next block in one pass,
                  the last in the type of x or in 8 bits with scales, and the gradients of all of it
* quantize_rows   rows to 8-bit integers with a scale for each
* int8_matmul     the product of 8-bit integers with a scale for each token and each channel
* adjust_logits   penalties for repeated tokens, biases and grammar masks

`run` computes them in their plain form (elementary torch operations in 32 bits, each output rounded once),
or, where `own` is true, by the library's kernels.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}

_handles = []


def _library():
    """The one library handle that a program keeps."""
    if not _handles:
        from async_pipelines_gb300 import gemm_ws
        _handles.append(gemm_ws.GemmWS(torch.cuda.current_device()))
    return _handles[0]


# ------------------------------------------------------------------ cases

def _block(name, T, H, dtype, form, gate, post=True, alpha=1.0, pad=0):
    return {"name": name, "op": "block", "T": T, "H": H, "dtype": dtype, "form": form, "gate": gate, "post": post,
            "alpha": alpha, "pad": pad}


def _product(name, M, K, N, source, out, bias=False):
    return {"name": name, "op": "product", "M": M, "K": K, "N": N, "source": source, "out": out, "bias": bias}


def _quantize(name, T, H, dtype, pad=0):
    return {"name": name, "op": "quantize", "T": T, "H": H, "dtype": dtype, "pad": pad}


def _logits(name, rows, vocab, dtype, out, history, prompt, penalties, biases, allowed):
    return {"name": name, "op": "logits", "rows": rows, "vocab": vocab, "dtype": dtype, "out": out, "history": history,
            "prompt": prompt, "penalties": penalties, "biases": biases, "allowed": allowed}


def listed():
    return [
        # one decoded token between two blocks, before a product in e4m3
        _block("block_token_8bit", 1, 8192, "bf16", "row8", "cols"),
        # odd sizes and rows that are not aligned, forward and backward
        _block("block_train_odd", 999, 1001, "f16", "train", "cols", pad=2),
        # a ragged number of tokens whose gates are computed for each of them, without a norm after the block
        _block("block_train_gated", 5000, 4096, "bf16", "train", "rows", post=False),
        # a training step of 8192 tokens, forward and backward, a gate for each channel and a scaled residual
        _block("block_train_large", 8192, 8192, "bf16", "train", "cols", alpha=0.9),
        # one token's logits over a large vocabulary
        _product("int8_token", 1, 4096, 131072, "given", "f32"),
        # a decode batch: the norms around a block in 8-bit integers, and the projection that takes them
        _product("int8_decode", 64, 8192, 8192, "block", "bf16"),
        # a ragged prompt quantised by the step, with a bias
        _product("int8_prompt_ragged", 5000, 4000, 3000, "rows", "f16", bias=True),
        # a large projection
        _product("int8_large", 8192, 8192, 8192, "given", "bf16"),
        # what has no norm before it: a large activation to 8-bit integers
        _quantize("quantize_large", 8192, 8192, "bf16"),
        # one sequence's logits with all that can be asked for
        _logits("logits_token", 1, 131072, "bf16", "f32", 1500, 700, True, 40, 0.9),
        # few rows of an odd vocabulary with a long history, penalties alone
        _logits("logits_long_history", 7, 50001, "f16", "f16", 32768, 20000, True, 0, 0.0),
        # a decode batch of 256, each in a grammar that allows few tokens
        _logits("logits_batch", 256, 131072, "f32", "f32", 2048, 900, True, 16, 0.02),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("block", "block", "product", "product", "quantize", "logits"))
    if op == "product":
        while True:
            M, K, N = _log(rng, 1, 8192), _log(rng, 64, 16384), _log(rng, 64, 131072)
            if rng.random() < 0.5:
                K = max(64, K // 64 * 64)
            if M * K * N <= 8192 ** 3 and M * N <= 8192 * 8192 and K * N <= 4096 * 131072:
                break
        c = _product("", M, K, N, rng.choice(("given", "given", "rows", "block")), rng.choice(("bf16", "bf16", "f16", "f32")),
                     rng.random() < 0.3)
    elif op == "logits":
        rows, vocab = _log(rng, 1, 512), _log(rng, 1000, 262144)
        while rows * vocab > 256 * 131072:
            rows = (rows + 1) // 2
        dtype = rng.choice(("bf16", "f16", "f32"))
        history = rng.choice((0, _log(rng, 1, 32768), _log(rng, 1, 32768)))
        while rows * history > 256 * 8192:
            history //= 2
        c = _logits("", rows, vocab, dtype, rng.choice((dtype, "f32")), history, int(rng.random() * history),
                    history > 0, rng.choice((0, 1, 40, 300)), rng.choice((0.0, 0.02, 0.9)))
    else:
        T, H = _log(rng, 1, 16384), _log(rng, 64, 16384)
        if rng.random() < 0.5:
            H = max(64, H // 8 * 8)
        while T * H > 8192 * 8192:
            T = (T + 1) // 2
        dtype, pad = rng.choice(("bf16", "bf16", "f16", "f32")), rng.choice((0, 0, 3, 8))
        if op == "quantize":
            c = _quantize("", T, H, dtype, pad)
        else:
            c = _block("", T, H, dtype, rng.choice(("infer", "row8", "group8", "train", "train")),
                       rng.choice(("none", "cols", "cols", "rows")), rng.random() < 0.8, rng.choice((1.0, 0.9, 2.6)), pad)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _rows(T, H, pad, dtype, gen, scale=1.0):
    """T rows of H values, `pad` more between one row and the next."""
    buf = torch.randn(T, H + pad, device="cuda", dtype=torch.float32, generator=gen)
    buf *= scale
    return buf.to(dtype)[:, :H]


def _channels(H, gen):
    """Some channels of a residual stream are larger than others."""
    return torch.exp(0.7 * torch.randn(H, device="cuda", generator=gen))


def _block_inputs(s, T, H, dtype, gate, post, pad, gen):
    s["x"] = _rows(T, H, pad, dtype, gen, 2.0)
    s["res"] = _rows(T, H, pad, dtype, gen, 3.0 * _channels(H + pad, gen))
    s["w"] = (1.0 + 0.2 * torch.randn(H, device="cuda", generator=gen)).to(dtype)
    s["post"] = (1.0 + 0.2 * torch.randn(H, device="cuda", generator=gen)).to(dtype) if post else None
    s["gate"] = None
    if gate == "cols":
        s["gate"] = (0.5 + 0.2 * torch.randn(H, device="cuda", generator=gen)).to(dtype)
    elif gate == "rows":
        s["gate"] = torch.sigmoid(torch.randn(T, H, device="cuda", generator=gen)).to(dtype)
    s["h"] = torch.empty(T, H, device="cuda", dtype=dtype)


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    s = {"case": case}
    return {"block": _prepare_block, "product": _prepare_product, "quantize": _prepare_quantize,
            "logits": _prepare_logits}[case["op"]](s, case, gen)


def _prepare_block(s, case, gen):
    T, H, dtype, pad = case["T"], case["H"], TYPES[case["dtype"]], case["pad"]
    _block_inputs(s, T, H, dtype, case["gate"], case["post"], pad, gen)
    if case["form"] in ("row8", "group8"):
        groups = 1 if case["form"] == "row8" else (H + 127) // 128
        s["y"] = torch.empty(T, H, device="cuda", dtype=torch.float8_e4m3fn)
        s["scales"] = torch.empty(T, groups, device="cuda")
    else:
        s["y"] = torch.empty(T, H, device="cuda", dtype=dtype)
    if case["form"] == "train":
        s["post_rstd"] = torch.empty(T, device="cuda") if case["post"] else None
        s["rstd"] = torch.empty(T, device="cuda")
        s["dy"] = _rows(T, H, pad, dtype, gen)
        s["dh"] = _rows(T, H, pad, dtype, gen, 0.5)
        s["dx"], s["dres"] = (torch.empty(T, H, device="cuda", dtype=dtype) for _ in range(2))
        s["dw"] = torch.empty_like(s["w"])
        s["dpost"] = torch.empty_like(s["post"]) if case["post"] else None
        s["dgate"] = torch.empty_like(s["gate"]) if s["gate"] is not None else None
    return s


def _prepare_product(s, case, gen):
    M, K, N = case["M"], case["K"], case["N"]
    # weights of about 1 / sqrt(K), quantised once by channels; rows on 16-byte boundaries
    pitch = (K + 15) // 16 * 16
    s["w8"] = torch.zeros(N, pitch, device="cuda", dtype=torch.int8)[:, :K]
    s["ws"] = torch.empty(N, device="cuda")
    step = max(1, (1 << 28) // K)
    for a in range(0, N, step):
        w = torch.randn(min(step, N - a), K, device="cuda", generator=gen)
        w *= torch.exp(0.3 * torch.randn(len(w), 1, device="cuda", generator=gen)) / math.sqrt(K)
        scale = w.abs().amax(1) / 127.0
        s["ws"][a:a + step] = scale
        s["w8"][a:a + step] = (w / scale[:, None]).round().to(torch.int8)
    s["bias"] = 0.5 * torch.randn(N, device="cuda", generator=gen) if case["bias"] else None
    s["d"] = torch.empty(M, N, device="cuda", dtype=TYPES[case["out"]])
    if case["source"] == "block":
        _block_inputs(s, M, K, torch.bfloat16, "cols", True, 0, gen)
    else:
        s["x"] = _rows(M, K, 0, torch.bfloat16, gen, _channels(K, gen))
    if case["source"] == "given":
        x = s.pop("x").float()
        s["as"] = x.abs().amax(1) / 127.0
        s["a8"] = (x / s["as"][:, None]).round().to(torch.int8)
    else:
        s["as"] = torch.empty(M, device="cuda")
        s["a8"] = torch.empty(M, K, device="cuda", dtype=torch.int8)
    return s


def _prepare_quantize(s, case, gen):
    T, H = case["T"], case["H"]
    s["x"] = _rows(T, H, case["pad"], TYPES[case["dtype"]], gen, _channels(H + case["pad"], gen))
    s["a8"] = torch.empty(T, H, device="cuda", dtype=torch.int8)
    s["as"] = torch.empty(T, device="cuda")
    return s


def _prepare_logits(s, case, gen):
    rows, vocab, S = case["rows"], case["vocab"], case["history"]
    s["z"] = _rows(rows, vocab, 0, TYPES[case["dtype"]], gen, 3.0)
    s["out"] = torch.empty(rows, vocab, device="cuda", dtype=TYPES[case["out"]])
    s["tokens"] = s["lengths"] = s["prompts"] = s["allowed"] = s["ids"] = s["values"] = None
    s["rep"] = s["freq"] = s["pres"] = None
    if S > 0:
        # words are frequent by their rank, so that some come back often
        u = torch.rand(rows, S, device="cuda", generator=gen, dtype=torch.float64)
        s["tokens"] = (vocab ** u - 1.0).long().clamp_(0, vocab - 1)
        s["lengths"] = (S - torch.randint(0, S // 4 + 1, (rows,), device="cuda", generator=gen)).int()
        s["prompts"] = torch.minimum(torch.full((rows,), case["prompt"], device="cuda", dtype=torch.int32), s["lengths"])
    if case["penalties"]:
        s["rep"] = 1.0 + 0.3 * torch.rand(rows, device="cuda", generator=gen)
        s["freq"] = torch.rand(rows, device="cuda", generator=gen) - 0.2
        s["pres"] = torch.rand(rows, device="cuda", generator=gen)
    if case["biases"]:
        s["ids"] = torch.randint(vocab, (rows, case["biases"]), device="cuda", generator=gen)
        s["values"] = 5.0 * torch.randn(rows, case["biases"], device="cuda", generator=gen)
    if case["allowed"]:
        words = (vocab + 31) // 32
        s["allowed"] = torch.zeros(rows, words, device="cuda", dtype=torch.int32)
        for bit in range(32):
            yes = torch.rand(rows, words, device="cuda", generator=gen) < case["allowed"]
            s["allowed"] |= yes.int() << bit
    return s


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"block": _own_block, "product": _own_product, "quantize": _own_quantize, "logits": _own_logits}[op](s)
    return {"block": _plain_block, "product": _plain_product, "quantize": _plain_quantize, "logits": _plain_logits}[op](s)


def _given(**outputs):
    return {k: v for k, v in outputs.items() if v is not None}


def _own_block(s):
    g, c = _library(), s["case"]
    train = c["form"] == "train"
    g.block_norm(s["x"], s["res"], s["w"], s["y"], post_weight=s["post"], gate=s["gate"], alpha=c["alpha"], h=s["h"],
                 post_rstd=s["post_rstd"] if train else None, rstd=s["rstd"] if train else None, scales=s.get("scales"), eps=EPS)
    out = _given(y=s["y"], h=s["h"], scales=s.get("scales"))
    if train:
        g.block_norm_backward(s["dy"], s["x"], s["h"], s["w"], s["rstd"], s["dx"], s["dres"], post_weight=s["post"],
                              post_rstd=s["post_rstd"], gate=s["gate"], alpha=c["alpha"], dh=s["dh"], dweight=s["dw"],
                              dpost_weight=s["dpost"], dgate=s["dgate"])
        out |= _given(post_rstd=s["post_rstd"], rstd=s["rstd"], dx=s["dx"], dres=s["dres"], dw=s["dw"], dpost=s["dpost"],
                      dgate=s["dgate"])
    return out


def _own_product(s):
    g, source = _library(), s["case"]["source"]
    out = {}
    if source == "block":
        g.block_norm(s["x"], s["res"], s["w"], s["a8"], post_weight=s["post"], gate=s["gate"], h=s["h"], scales=s["as"], eps=EPS)
        out = {"h": s["h"], "as": s["as"]}
    elif source == "rows":
        g.quantize_rows(s["x"], s["a8"], s["as"])
        out = {"a8": s["a8"], "as": s["as"]}
    g.int8_matmul(s["a8"], s["w8"], s["as"], s["ws"], s["d"], bias=s["bias"])
    return out | {"d": s["d"]}


def _own_quantize(s):
    _library().quantize_rows(s["x"], s["a8"], s["as"])
    return {"a8": s["a8"], "as": s["as"]}


def _own_logits(s):
    _library().adjust_logits(s["z"], s["out"], tokens=s["tokens"], lengths=s["lengths"], prompt_lengths=s["prompts"],
                             repetition=s["rep"], frequency=s["freq"], presence=s["pres"], bias_tokens=s["ids"],
                             bias_values=s["values"], allowed=s["allowed"])
    return {"out": s["out"]}


# ------------------------------------------------------------------ plain forms

def _plain_join(s, alpha):
    """(n, post_rstd, h) of a block's norm, gate and residual, in 32 bits."""
    x = s["x"].float()
    r1 = ((x * x).mean(1, keepdim=True) + EPS).rsqrt() if s["post"] is not None else None
    n = x if r1 is None else x * r1
    b = n if r1 is None else n * s["post"].float()
    if s["gate"] is not None:
        b = b * s["gate"].float()
    return n, r1, alpha * s["res"].float() + b


def _plain_block(s):
    c, dtype = s["case"], s["x"].dtype
    T, H, w = c["T"], c["H"], s["w"].float()
    n, r1, h = _plain_join(s, c["alpha"])
    r2 = ((h * h).mean(1, keepdim=True) + EPS).rsqrt()
    y = h * r2 * w
    out = {"h": h.to(dtype)}
    if c["form"] in ("row8", "group8"):
        group = H if c["form"] == "row8" else 128
        groups = (H + group - 1) // group
        padded = torch.zeros(T, groups * group, device="cuda")
        padded[:, :H] = y
        padded = padded.view(T, groups, group)
        scales = (padded.abs().amax(2) / E4M3_MAX).clamp(min=2.0 ** -126)
        out["y"] = (padded / scales[:, :, None]).view(T, -1)[:, :H].to(torch.float8_e4m3fn)
        out["scales"] = scales
        return out
    out["y"] = y.to(dtype)
    if c["form"] == "train":
        del h, y
        dy, nh = s["dy"].float(), out["h"].float() * r2
        out["dw"] = (dy * nh).sum(0).to(dtype)
        a = dy * w
        g = s["dh"].float() + r2 * (a - nh * (a * nh).mean(1, keepdim=True))
        del dy, nh, a
        out["dres"] = (c["alpha"] * g).to(dtype)
        post = None if s["post"] is None else s["post"].float()
        if s["gate"] is not None:
            db = g * (n if post is None else n * post)
            out["dgate"] = (db if c["gate"] == "rows" else db.sum(0)).to(dtype)
            g = g * s["gate"].float()
        if post is not None:
            out["dpost"] = (g * n).sum(0).to(dtype)
            a = g * post
            g = r1 * (a - n * (a * n).mean(1, keepdim=True))
            out["post_rstd"] = r1[:, 0]
        out |= {"dx": g.to(dtype), "rstd": r2[:, 0]}
    return out


def _plain_rows8(x):
    """Rows of 32-bit values as whole numbers from -127 to 127, and their scales."""
    top = x.abs().amax(1)
    # by a tensor: a division by a number is a product with its inverse
    scale = (top / torch.full_like(top, 127.0)).clamp(min=2.0 ** -126)
    return (x / scale[:, None]).round(), scale


def _plain_product(s):
    source, out = s["case"]["source"], {}
    if source == "block":
        _, _, h = _plain_join(s, 1.0)
        a, scale = _plain_rows8(h * ((h * h).mean(1, keepdim=True) + EPS).rsqrt() * s["w"].float())
        out = {"h": h.to(s["x"].dtype), "as": scale}
    elif source == "rows":
        a, scale = _plain_rows8(s["x"].float())
        out = {"a8": a.to(torch.int8), "as": scale}
    else:
        a, scale = s["a8"].float(), s["as"]
    d = (a @ s["w8"].float().T) * scale[:, None] * s["ws"]
    if s["bias"] is not None:
        d += s["bias"]
    return out | {"d": d.to(s["d"].dtype)}


def _plain_quantize(s):
    a, scale = _plain_rows8(s["x"].float())
    return {"a8": a.to(torch.int8), "as": scale}


def _plain_logits(s):
    c = s["case"]
    z = s["z"].float()
    if s["tokens"] is not None:
        at = torch.arange(c["history"], device="cuda")[None, :]
        inside = at < s["lengths"][:, None]
        new = inside & (at >= s["prompts"][:, None])
        seen = torch.zeros(c["rows"], c["vocab"], device="cuda").scatter_add_(1, s["tokens"], inside.float()) > 0
        count = torch.zeros(c["rows"], c["vocab"], device="cuda").scatter_add_(1, s["tokens"], new.float())
        rep = s["rep"][:, None]
        z = torch.where(seen, torch.where(z > 0, z / rep, z * rep), z)
        z = z - (s["freq"][:, None] * count + s["pres"][:, None] * (count > 0))
    if s["ids"] is not None:
        z = z.scatter_add(1, s["ids"], s["values"])
    if s["allowed"] is not None:
        v = torch.arange(c["vocab"], device="cuda")
        z = torch.where((s["allowed"][:, v >> 5] >> (v & 31)) & 1 > 0, z, -math.inf)
    return {"out": z.to(s["out"].dtype)}


# ------------------------------------------------------------------ in 64 bits

def _exact_join(s, alpha):
    x, h = s["x"].double(), alpha * s["res"].double()
    r = None
    if s["post"] is not None:
        r = 1.0 / torch.sqrt(torch.einsum("ij,ij->i", x, x) / x.shape[1] + EPS)
        x = torch.einsum("ij,i,j->ij", x, r, s["post"].double())
    return r, h + (x if s["gate"] is None else x * s["gate"].double())


def _exact_norm(h, w):
    r = 1.0 / torch.sqrt(torch.einsum("ij,ij->i", h, h) / h.shape[1] + EPS)
    return r, torch.einsum("ij,i,j->ij", h, r, w.double())


def exact(case, seed):
    s = prepare(case, seed)
    return {"block": _exact_block, "product": _exact_product, "quantize": _exact_quantize, "logits": _exact_logits}[case["op"]](case, s)


def _exact_block(case, s):
    H = case["H"]
    r1, h = _exact_join(s, case["alpha"])
    r2, y = _exact_norm(h, s["w"])
    out = {"h": h}
    if case["form"] in ("row8", "group8"):
        size = H if case["form"] == "row8" else 128
        scales, values = [], []
        for a in range(0, H, size):
            part = y[:, a:a + size]
            scale = (part.abs().max(dim=1).values / E4M3_MAX).clamp(min=2.0 ** -126)
            scales.append(scale)
            values.append(part / scale[:, None])
        return out | {"y": torch.cat(values, 1), "scales": torch.stack(scales, 1)}
    out["y"] = y
    if case["form"] == "train":
        # the backward pass is given h in its own type
        stored = h.to(s["x"].dtype).double()
        dy, w = s["dy"].double(), s["w"].double()
        dot = torch.einsum("ij,ij,j->i", dy, stored, w)
        g = s["dh"].double() + dy * w * r2[:, None] - stored * (dot * r2 ** 3 / H)[:, None]
        out |= {"rstd": r2, "dres": case["alpha"] * g, "dw": torch.einsum("ij,ij,i->j", dy, stored, r2)}
        x = s["x"].double()
        gate = torch.ones(1, H, device="cuda", dtype=torch.float64) if s["gate"] is None else s["gate"].double().view(-1, H)
        one = torch.ones(H, device="cuda", dtype=torch.float64)
        post = one if s["post"] is None else s["post"].double()
        r = torch.ones(len(x), device="cuda", dtype=torch.float64) if r1 is None else r1
        if s["gate"] is not None:
            if case["gate"] == "rows":
                out["dgate"] = g * x * r[:, None] * post
            else:
                out["dgate"] = torch.einsum("ij,ij,i->j", g, x, r) * post
        db = g * gate
        if r1 is None:
            out["dx"] = db
        else:
            out["post_rstd"] = r1
            out["dpost"] = torch.einsum("ij,ij,i->j", db, x, r1)
            dot = torch.einsum("ij,ij,j->i", db, x, post)
            out["dx"] = db * post * r1[:, None] - x * (dot * r1 ** 3 / H)[:, None]
    return out


def _exact_product(case, s):
    out = {}
    if case["source"] == "given":
        a, scale = s["a8"].double(), s["as"].double()
    else:
        if case["source"] == "block":
            _, h = _exact_join(s, 1.0)
            _, y = _exact_norm(h, s["w"])
            out = {"h": h}
        else:
            y = s["x"].double()
        # the scale is held in 32 bits
        scale = (y.abs().max(dim=1).values / 127.0).clamp(min=2.0 ** -126).float().double()
        a = torch.round(y / scale[:, None])
        out["as"] = scale
    parts = []
    step = max(1, (1 << 28) // case["K"])
    for k in range(0, case["N"], step):
        parts.append((a @ s["w8"][k:k + step].double().T) * scale[:, None] * s["ws"][k:k + step].double())
        if s["bias"] is not None:
            parts[-1] += s["bias"][k:k + step].double()
    return out | {"d": torch.cat(parts, 1)}


def _exact_quantize(case, s):
    # whole numbers have no 64-bit form of their own: they are what their 32-bit scale makes them
    return {"as": (s["x"].double().abs().max(dim=1).values / 127.0).clamp(min=2.0 ** -126)}


def _exact_logits(case, s):
    rows = []
    for r in range(case["rows"]):
        z = s["z"][r].double()
        if s["tokens"] is not None:
            n, p = int(s["lengths"][r]), int(s["prompts"][r])
            said = torch.bincount(s["tokens"][r, :n], minlength=case["vocab"])
            new = torch.bincount(s["tokens"][r, p:n], minlength=case["vocab"]).double()
            rep, freq, pres = (s[k][r].double() for k in ("rep", "freq", "pres"))
            known = said > 0
            z[known] = torch.where(z[known] > 0, z[known] / rep, z[known] * rep)
            z -= freq * new + pres * new.clamp(max=1.0)
        if s["ids"] is not None:
            z.index_add_(0, s["ids"][r], s["values"][r].double())
        if s["allowed"] is not None:
            bits = torch.stack([s["allowed"][r] >> b & 1 for b in range(32)], 1).flatten()[:case["vocab"]]
            z[bits == 0] = -math.inf
        rows.append(z)
    return {"out": torch.stack(rows)}


# ------------------------------------------------------------------ work

def work(case):
    if case["op"] == "product":
        M, K, N = case["M"], case["K"], case["N"]
        read = {"given": M * K + 4 * M, "rows": 2 * M * K, "block": 4 * M * K + 6 * K}[case["source"]]
        wrote = {"given": 0, "rows": M * K + 4 * M, "block": 2 * M * K + 4 * M}[case["source"]]
        product = N * K + 4 * N * (2 if case["bias"] else 1) + M * N * TYPES[case["out"]].itemsize
        return {"bytes": read + wrote + product, "flops": 2 * M * K * N + {"given": 0, "rows": 3, "block": 12}[case["source"]] * M * K}
    if case["op"] == "quantize":
        n = case["T"] * case["H"]
        return {"bytes": n * TYPES[case["dtype"]].itemsize + n + 4 * case["T"], "flops": 3 * n}
    if case["op"] == "logits":
        rows, vocab = case["rows"], case["vocab"]
        each = vocab * (TYPES[case["dtype"]].itemsize + TYPES[case["out"]].itemsize) + 8 * case["history"] + 12 * case["biases"]
        if case["allowed"]:
            each += (vocab + 31) // 32 * 4
        return {"bytes": rows * each, "flops": rows * (vocab + 6 * case["history"] + case["biases"])}
    T, H = case["T"], case["H"]
    size = TYPES[case["dtype"]].itemsize
    n = T * H
    vectors = (1 + case["post"] + (case["gate"] == "cols")) * H * size
    gates = n if case["gate"] == "rows" else 0
    forward = 3 * n * size + gates * size + vectors   # x, residual, h
    if case["form"] == "infer":
        return {"bytes": forward + n * size, "flops": 11 * n}
    if case["form"] in ("row8", "group8"):
        groups = 1 if case["form"] == "row8" else (H + 127) // 128
        return {"bytes": forward + n + 4 * T * groups, "flops": 13 * n}
    # forward: y and the statistics too; backward: dy, dh, x, h and the gates in, dx, dres and the gates' gradients out
    stats = 4 * T * (1 + case["post"])
    back = 6 * n * size + 2 * gates * size + 2 * vectors + stats
    return {"bytes": forward + n * size + stats + back, "flops": 38 * n}
