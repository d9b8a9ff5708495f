"""Cases of the language-model operators beside the GEMM: what they are given, what they return, and their plain forms.

Three operators that sit around the library's matrix product in the last part of a training step or of a
scoring step, as methods of `gemm_ws.GemmWS`:

* dropout            y = keep * x / (1 - p), the mask drawn from a counter and never stored
* add_rms_norm       h = residual + dropout(x), y = weight * h / rms(h), in the type of x or in 8 bits with
                     scales, and its gradients
* linear cross entropy  the softmax cross entropy of x @ weight^T over a vocabulary, and its gradients,
                     without the logits ever being held

`run` computes them in their plain form (elementary torch operations in 32 bits, each output rounded once),
or, where `own` is true, by the library's kernels.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
IGNORED = -100

_handles = []


def _library():
    """The one library handle that a program keeps."""
    if not _handles:
        from async_pipelines_gb300 import gemm_ws
        _handles.append(gemm_ws.GemmWS(torch.cuda.current_device()))
    return _handles[0]


# ------------------------------------------------------------------ cases

def _loss(name, T, H, V, train, ignored=0.0, pad=0):
    return {"name": name, "op": "loss", "T": T, "H": H, "V": V, "train": train, "ignored": ignored, "pad": pad}


def _norm(name, T, H, dtype, form, p=0.0, pad=0):
    return {"name": name, "op": "norm", "T": T, "H": H, "dtype": dtype, "form": form, "p": p, "pad": pad}


def _dropout(name, T, H, dtype, p, pad=0):
    return {"name": name, "op": "dropout", "T": T, "H": H, "dtype": dtype, "p": p, "pad": pad}


def listed():
    return [
        # the log-probability of one generated token over a large vocabulary: the weight is read once
        _loss("loss_score_token", 1, 4096, 131072, False),
        # scoring a short answer; a length that fills no tile
        _loss("loss_score_answer", 61, 8192, 32768, False),
        # a small model's step, where launches and waits count; a third of the tokens is prompt or padding
        _loss("loss_train_small", 256, 256, 1000, True, ignored=0.33),
        # ragged in every size, with the hidden states a slice of a wider buffer
        _loss("loss_train_ragged", 5000, 3000, 50001, True, ignored=0.1, pad=40),
        # a training step of a large vocabulary
        _loss("loss_train_large", 4096, 4096, 131072, True),
        # one decoded token: the norm before a product in 8 bits
        _norm("norm_token_8bit", 1, 8192, "bf16", "row8"),
        # a decode batch of 64 sequences
        _norm("norm_decode", 64, 4096, "bf16", "infer"),
        # a ragged prompt, 8 bits with a scale for each 128 columns
        _norm("norm_prompt_8bit", 5000, 4096, "bf16", "group8"),
        # odd sizes and rows that are not aligned, forward and backward
        _norm("norm_train_odd", 999, 1001, "f16", "train", pad=2),
        # a training step of 8192 tokens with dropout, forward and backward
        _norm("norm_train_large", 8192, 8192, "bf16", "train", p=0.1),
        # dropout of a small activation, forward and backward
        _dropout("dropout_small", 256, 256, "bf16", 0.5),
        # dropout of a large activation, forward and backward
        _dropout("dropout_large", 8192, 8192, "bf16", 0.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("loss", "loss", "norm", "norm", "dropout"))
    if op == "loss":
        while True:
            T, H, V = _log(rng, 1, 8192), 8 * _log(rng, 8, 1024), _log(rng, 100, 131072)
            if T * H * V <= 4096 * 4096 * 131072 and T * V <= 4096 * 131072:
                break
        c = _loss("", T, H, V, rng.random() < 0.6, rng.choice((0.0, 0.0, 0.25, 0.9)), 8 * rng.choice((0, 0, 1, 5)))
    else:
        T, H = _log(rng, 1, 16384), _log(rng, 64, 16384)
        if rng.random() < 0.5:
            H = max(64, H // 8 * 8)
        while T * H > 8192 * 8192:
            T = (T + 1) // 2
        dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
        pad = rng.choice((0, 0, 3, 8))
        if op == "norm":
            form = rng.choice(("infer", "row8", "group8", "train", "train"))
            c = _norm("", T, H, dtype, form, rng.choice((0.0, 0.1, 0.35)) if form == "train" else 0.0, pad)
        else:
            c = _dropout("", T, H, dtype, rng.choice((0.0, 0.1, 0.3, 0.5)), pad)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs

def _rows(T, H, pad, dtype, gen, scale=1.0):
    """T rows of H values, `pad` more between one row and the next."""
    buf = torch.randn(T, H + pad, device="cuda", dtype=torch.float32, generator=gen)
    buf *= scale
    return buf.to(dtype)[:, :H]


def prepare(case, seed):
    gen = torch.Generator("cuda").manual_seed(seed)
    T, H = case["T"], case["H"]
    s = {"case": case}
    if case["op"] == "loss":
        V, bf16 = case["V"], torch.bfloat16
        # logits of about N(0, 1.5^2), the target's raised by 0 to 14: from tokens that the model does not
        # expect to tokens that it is sure of
        w = torch.randn(V, H, device="cuda", dtype=bf16, generator=gen)
        w *= 1.5 / math.sqrt(H)
        t = torch.randint(V, (T,), device="cuda", generator=gen)
        up = torch.rand(T, 1, device="cuda", generator=gen) * (14.0 / 2.25)
        x = torch.randn(T, H + case["pad"], device="cuda", generator=gen)
        x[:, :H] += up * w[t].float()
        s["x"], s["w"] = x.to(bf16)[:, :H], w
        skip = torch.rand(T, device="cuda", generator=gen) < case["ignored"]
        s["t"] = torch.where(skip, torch.full_like(t, IGNORED), t)
        s["loss"] = torch.empty(T, device="cuda")
        s["lse"] = torch.empty(T, device="cuda")
        s["mean"] = torch.empty(2, device="cuda")
        if case["train"]:
            s["dx"] = torch.empty(T, H, device="cuda", dtype=bf16)
            s["dw"] = torch.empty(V, H, device="cuda", dtype=bf16)
        return s
    dtype, pad = TYPES[case["dtype"]], case["pad"]
    s["rng"] = torch.tensor([seed * 7919 + 12345, (1 << 33) + seed], device="cuda", dtype=torch.int64)
    s["x"] = _rows(T, H, pad, dtype, gen)
    if case["op"] == "dropout":
        s["dy"] = _rows(T, H, pad, dtype, gen)
        s["y"] = torch.empty(T, H, device="cuda", dtype=dtype)
        s["dx"] = torch.empty(T, H, device="cuda", dtype=dtype)
        return s
    # a residual stream some times larger than what is added to it, with a few large channels
    channel = torch.exp(0.7 * torch.randn(H + pad, device="cuda", generator=gen))
    s["res"] = _rows(T, H, pad, dtype, gen, 3.0 * channel)
    s["w"] = (1.0 + 0.2 * torch.randn(H, device="cuda", generator=gen)).to(dtype)
    s["h"] = torch.empty(T, H, device="cuda", dtype=dtype)
    if case["form"] in ("row8", "group8"):
        groups = 1 if case["form"] == "row8" else (H + 127) // 128
        s["y"] = torch.empty(T, H, device="cuda", dtype=torch.float8_e4m3fn)
        s["scales"] = torch.empty(T, groups, device="cuda")
    else:
        s["y"] = torch.empty(T, H, device="cuda", dtype=dtype)
    if case["form"] == "train":
        s["rstd"] = torch.empty(T, device="cuda")
        s["dy"] = _rows(T, H, pad, dtype, gen)
        s["dh"] = _rows(T, H, pad, dtype, gen, 0.5)
        s["dx"] = torch.empty(T, H, device="cuda", dtype=dtype)
        s["dres"] = torch.empty(T, H, device="cuda", dtype=dtype)
        s["dw"] = torch.empty(H, device="cuda", dtype=dtype)
    return s


EPS = 1e-6


# ------------------------------------------------------------------ one pass

def run(s):
    op = s["case"]["op"]
    if own:
        return {"loss": _own_loss, "norm": _own_norm, "dropout": _own_dropout}[op](s)
    return {"loss": _plain_loss, "norm": _plain_norm, "dropout": _plain_dropout}[op](s)


def _own_loss(s):
    g = _library()
    g.linear_cross_entropy(s["x"], s["w"], s["t"], s["loss"], s["lse"], mean=s["mean"], ignore_index=IGNORED)
    out = {"loss": s["loss"], "lse": s["lse"], "mean": s["mean"]}
    if s["case"]["train"]:
        # the gradient of the mean: each counted token's share is mean[1] = 1 / count
        g.linear_cross_entropy_backward(s["x"], s["w"], s["t"], s["lse"], s["mean"][1:], dx=s["dx"],
                                        dweight=s["dw"], ignore_index=IGNORED)
        out |= {"dx": s["dx"], "dw": s["dw"]}
    return out


def _own_norm(s):
    g, c = _library(), s["case"]
    p = c["p"]
    if c["form"] != "train":
        g.add_rms_norm(s["x"], s["w"], s["y"], residual=s["res"], h=s["h"], scales=s.get("scales"), eps=EPS)
        out = {"y": s["y"], "h": s["h"]}
        if "scales" in s:
            out["scales"] = s["scales"]
        return out
    g.add_rms_norm(s["x"], s["w"], s["y"], residual=s["res"], h=s["h"], rstd=s["rstd"], eps=EPS, p=p,
                   rng=s["rng"])
    g.add_rms_norm_backward(s["dy"], s["h"], s["w"], s["rstd"], s["dx"], s["dw"], dh=s["dh"],
                            dresidual=s["dres"] if p > 0 else None, p=p, rng=s["rng"])
    out = {"y": s["y"], "h": s["h"], "rstd": s["rstd"], "dx": s["dx"], "dw": s["dw"]}
    if p > 0:
        out["dres"] = s["dres"]
    return out


def _own_dropout(s):
    g, p = _library(), s["case"]["p"]
    g.dropout(s["x"], s["y"], p, s["rng"])
    g.dropout(s["dy"], s["dx"], p, s["rng"])
    return {"y": s["y"], "dx": s["dx"]}


# ------------------------------------------------------------------ plain forms

def _plain_loss(s):
    x, w, t = s["x"].float(), s["w"].float(), s["t"]
    z = x @ w.T
    top = z.amax(1, keepdim=True)
    lse = top + (z - top).exp().sum(1, keepdim=True).log()
    # an ignored token has no loss, no lse and no gradient: zeros
    counted = (t != IGNORED)[:, None]
    at = torch.where(counted, t[:, None], 0)
    lse = torch.where(counted, lse, 0.0)
    loss = torch.where(counted, lse - z.gather(1, at), 0.0)
    count = counted.sum()
    share = torch.where(count > 0, 1.0 / count.clamp(min=1), 0.0)
    out = {"loss": loss[:, 0], "lse": lse[:, 0], "mean": torch.stack((loss.sum() * share, share))}
    if s["case"]["train"]:
        g = torch.where(counted, z - lse, 0.0).exp_()
        g.scatter_add_(1, at, torch.full_like(lse, -1.0))
        g *= counted * share
        out["dx"] = (g @ w).to(torch.bfloat16)
        out["dw"] = (g.T @ x).to(torch.bfloat16)
    return out


def _philox(rng, T, H):
    """The 16-bit words of elements (row, column), T x H: Philox4x32 of ten rounds (Salmon et al., 2011), key
    the seed, counter offset + row * ceil(H / 8) + column / 8, whose 128 bits are eight words, lowest first."""
    low = 0xFFFFFFFF
    per_row = (H + 7) // 8
    c = rng[1] + torch.arange(T * per_row, device="cuda")
    a0, a1, a2, a3 = c & low, (c >> 32) & low, torch.zeros_like(c), torch.zeros_like(c)
    k0, k1 = rng[0] & low, (rng[0] >> 32) & low
    for _ in range(10):
        m0, m1 = a0 * 0xD2511F53, a2 * 0xCD9E8D57
        a0, a1, a2, a3 = ((m1 >> 32) & low) ^ a1 ^ k0, m1 & low, ((m0 >> 32) & low) ^ a3 ^ k1, m0 & low
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    words = torch.stack((a0, a1, a2, a3), 1)
    halves = torch.stack((words & 0xFFFF, words >> 16), 2)
    return halves.reshape(T, per_row * 8)[:, :H]


def _keep(rng, T, H, p):
    """What each element is multiplied by: 0 where its word is below p * 2^16, else the inverse of the share kept."""
    below = round(p * 65536)
    if below >= 65536:
        return torch.zeros(T, H, device="cuda")
    return (_philox(rng, T, H) >= below) * torch.tensor(65536.0 / (65536 - below), device="cuda")


def _plain_dropout(s):
    c = s["case"]
    keep = _keep(s["rng"], c["T"], c["H"], c["p"])
    return {"y": (s["x"].float() * keep).to(s["x"].dtype), "dx": (s["dy"].float() * keep).to(s["x"].dtype)}


def _plain_norm(s):
    c, dtype = s["case"], s["x"].dtype
    T, H = c["T"], c["H"]
    x, w = s["x"].float(), s["w"].float()
    keep = _keep(s["rng"], T, H, c["p"]) if c["p"] > 0 else None
    h = s["res"].float() + (x if keep is None else x * keep)
    rstd = ((h * h).mean(1, keepdim=True) + EPS).rsqrt()
    y = h * rstd * w
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
        n = out["h"].float() * rstd
        dy = s["dy"].float()
        a = dy * w
        dh = s["dh"].float() + rstd * (a - n * (a * n).mean(1, keepdim=True))
        out |= {"rstd": rstd[:, 0], "dx": (dh if keep is None else dh * keep).to(dtype), "dw": (dy * n).sum(0).to(dtype)}
        if keep is not None:
            out["dres"] = dh.to(dtype)
    return out


# ------------------------------------------------------------------ in 64 bits

def exact(case, seed):
    if case["op"] == "loss":
        return _exact_loss(case, seed)
    s = prepare(case, seed)
    T, H, p = case["T"], case["H"], case["p"]
    mask = None
    if p > 0:
        # the same generator, with each product put together from 16-bit halves
        def mul(a, b):
            al, ah, bl, bh = a % 65536, a // 65536, b % 65536, b // 65536
            mid = al * bh + (al * bl) // 65536
            mid2 = ah * bl + mid % 65536
            return ah * bh + mid // 65536 + mid2 // 65536, (mid2 % 65536) * 65536 + (al * bl) % 65536
        seed64, first = (int(v) for v in s["rng"].tolist())
        groups = -(-H // 8)
        n = torch.arange(T * groups, device="cuda") + first
        word = [n % 2 ** 32, n // 2 ** 32, n * 0, n * 0]
        key = [seed64 % 2 ** 32, seed64 // 2 ** 32]
        for _ in range(10):
            h0, l0 = mul(word[0], 0xD2511F53)
            h1, l1 = mul(word[2], 0xCD9E8D57)
            word = [h1 ^ word[1] ^ key[0], l1, h0 ^ word[3] ^ key[1], l0]
            key = [(key[0] + 0x9E3779B9) % 2 ** 32, (key[1] + 0xBB67AE85) % 2 ** 32]
        mask = torch.empty(T * groups, 8, device="cuda", dtype=torch.bool)
        for k in range(4):
            mask[:, 2 * k] = word[k] % 65536 >= round(p * 65536)
            mask[:, 2 * k + 1] = word[k] // 65536 >= round(p * 65536)
        mask = mask.view(T, groups * 8)[:, :H]
        share = 1.0 - round(p * 65536) / 65536.0

    def drop(v):
        return v if mask is None else torch.where(mask, v / share, torch.zeros_like(v))

    if case["op"] == "dropout":
        return {"y": drop(s["x"].double()), "dx": drop(s["dy"].double())}
    h = s["res"].double() + drop(s["x"].double())
    var = torch.einsum("ij,ij->i", h, h) / H
    r = 1.0 / torch.sqrt(var + EPS)
    w = s["w"].double()
    y = w * (h * r[:, None])
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
        dy = s["dy"].double()
        dot = torch.einsum("ij,ij,j->i", dy, stored, w)
        dh = s["dh"].double() + dy * w * r[:, None] - stored * (dot * r ** 3 / H)[:, None]
        out |= {"rstd": r, "dx": drop(dh), "dw": torch.einsum("ij,ij,i->j", dy, stored, r)}
        if mask is not None:
            out["dres"] = dh
    return out


def _exact_loss(case, seed):
    T, H, V = case["T"], case["H"], case["V"]
    if (6 if case["train"] else 2) * T * H * V > 1.4e13:
        return None   # over 20 seconds in 64 bits
    s = prepare(case, seed)
    x, w, t = s["x"].double(), s["w"].double(), s["t"]
    counted = t != IGNORED
    n = int(counted.sum())
    rows = max(1, (1 << 28) // V)
    lse, loss, dx = [], [], []
    dw = torch.zeros(V, H, device="cuda", dtype=torch.float64) if case["train"] else None
    for a in range(0, T, rows):
        z = x[a:a + rows] @ w.T
        lse.append(torch.where(counted[a:a + rows], torch.logsumexp(z, 1), 0.0))
        at = t[a:a + rows].clamp(min=0)
        k = torch.arange(len(at), device="cuda")
        loss.append(torch.where(counted[a:a + rows], lse[-1] - z[k, at], 0.0))
        if case["train"]:
            z -= lse[-1][:, None]
            z.masked_fill_(~counted[a:a + rows, None], -math.inf)
            z.exp_()
            z[k, at] -= counted[a:a + rows].double()
            z /= max(n, 1)
            dx.append(z @ w)
            dw.addmm_(z.T, x[a:a + rows])
    loss = torch.cat(loss)
    mean = torch.stack((loss.sum() / max(n, 1), torch.tensor(1.0 / n if n else 0.0, device="cuda", dtype=torch.float64)))
    out = {"loss": loss, "lse": torch.cat(lse), "mean": mean}
    return out | {"dx": torch.cat(dx), "dw": dw} if case["train"] else out


# ------------------------------------------------------------------ work

def work(case):
    T, H = case["T"], case["H"]
    if case["op"] == "loss":
        V = case["V"]
        given = 2 * T * H + 2 * V * H + 8 * T
        if case["train"]:
            # logits, gradient of x, gradient of the weight
            return {"bytes": given + 8 * T + 2 * T * H + 2 * V * H, "flops": 6 * T * H * V}
        return {"bytes": given + 8 * T, "flops": 2 * T * H * V}
    size = TYPES[case["dtype"]].itemsize
    n = T * H
    if case["op"] == "dropout":
        return {"bytes": 4 * n * size, "flops": 4 * n}
    forward = 3 * n * size + H * size   # x, residual, h
    if case["form"] == "infer":
        return {"bytes": forward + n * size, "flops": 6 * n}
    if case["form"] in ("row8", "group8"):
        groups = 1 if case["form"] == "row8" else (H + 127) // 128
        return {"bytes": forward + n + 4 * T * groups, "flops": 8 * n}
    # forward: y and rstd too; backward: dy, h, dh, rstd and the weight in, dx, (the residual's gradient) and dw out
    back = (5 if case["p"] > 0 else 4) * n * size + 4 * T + 2 * H * size
    return {"bytes": forward + n * size + 4 * T + back, "flops": 18 * n}
