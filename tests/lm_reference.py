"""Plain implementations in 64 bits of the language-model operators, for the tests.

They follow the formulas of include/gemm_ws_lm.h and share no code with the library.
"""
from __future__ import annotations

import torch

# Half the distance between neighbouring values near 1: a rounding moves a value by at most this share.
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}
# Half the distance between the smallest values of a type.
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
E4M3_UNIT, E4M3_TINY, E4M3_MAX = 2.0 ** -4, 2.0 ** -10, 448.0


def philox(counter, key):
    """Philox4x32-10: four 32-bit words of a 128-bit counter (low word first) and a 64-bit key."""
    c = [(counter >> (32 * i)) & 0xFFFFFFFF for i in range(4)]
    k0, k1 = key & 0xFFFFFFFF, key >> 32
    for _ in range(10):
        m0, m1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(m1 >> 32) ^ c[1] ^ k0, m1 & 0xFFFFFFFF, (m0 >> 32) ^ c[3] ^ k1, m0 & 0xFFFFFFFF]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return c


def keep_factor(rows, cols, p, rng):
    """rows x cols in 64 bits: 0 where an element is dropped, else what it is multiplied by."""
    below = round(p * 65536)
    if below == 0:
        return torch.ones(rows, cols, dtype=torch.float64)
    if below == 65536:
        return torch.zeros(rows, cols, dtype=torch.float64)
    seed, first = (int(v) & 0xFFFFFFFFFFFFFFFF for v in rng)
    groups = (cols + 7) // 8
    words = []
    for n in range(rows * groups):
        for w in philox((first + n) & 0xFFFFFFFFFFFFFFFF, seed):
            words += (w & 0xFFFF, w >> 16)
    words = torch.tensor(words).view(rows, groups * 8)[:, :cols]
    return (words >= below).double() * (65536.0 / (65536 - below))


def apply_keep(x, keep):
    """A dropped value is 0 whatever it was."""
    return torch.where(keep == 0, torch.zeros_like(x), x * keep)


def add_rms_norm(x, residual, weight, eps, keep=None):
    """h, rstd and y in 64 bits."""
    h = x.double() if keep is None else apply_keep(x.double(), keep)
    if residual is not None:
        h = h + residual.double()
    rstd = 1.0 / torch.sqrt((h * h).sum(1) / h.shape[1] + eps)
    return h, rstd, h * rstd[:, None] * weight.double()


def add_rms_norm_backward(dy, h, weight, rstd, dh=None, keep=None):
    """dx, dresidual, dweight, and the sums of magnitudes that their errors go by."""
    dy, h, w, r = dy.double(), h.double(), weight.double(), rstd.double()[:, None]
    a, n = dy * w, h * r
    c = (a * n).mean(1, keepdim=True)
    dres = r * (a - n * c)
    size = r * (a.abs() + n.abs() * (a * n).abs().mean(1, keepdim=True))
    if dh is not None:
        dres = dres + dh.double()
        size = size + dh.double().abs()
    dx = dres if keep is None else apply_keep(dres, keep)
    return dx, dres, (dy * n).sum(0), size, (dy * n).abs().sum(0)


def linear_cross_entropy(x, weight, target, ignore):
    """loss, lse and the mean over the counted tokens, in 64 bits."""
    z = x.double() @ weight.double().T
    counted = target != ignore
    lse = torch.where(counted, torch.logsumexp(z, 1), 0.0)
    at = torch.where(counted, target, 0)
    loss = torch.where(counted, lse - z.gather(1, at[:, None])[:, 0], 0.0)
    n = int(counted.sum())
    return loss, lse, float(loss.sum()) / max(n, 1)


def linear_cross_entropy_backward(x, weight, target, grad, ignore):
    """dx and dweight, and the sums of magnitudes that their errors go by."""
    x, w = x.double(), weight.double()
    counted = target != ignore
    x = torch.where(counted[:, None], x, 0.0)
    g = torch.softmax(x @ w.T, 1)
    g[torch.arange(len(target)), torch.where(counted, target, 0)] -= 1.0
    g = torch.where(counted[:, None], g * grad.double()[:, None], 0.0)
    return g @ w, g.T @ x, g.abs() @ w.abs(), g.abs().T @ x.abs()
