"""Plain 64-bit forms of the operators that train, balance and quantise, and the
error bounds their GPU tests use (CPU, torch float64).

Bounds count roundings as tests/decode_util.py does: U = 2^-24 for an fp32
operation, half a step of T for a rounding to T.
"""
import math

import torch

from tests.decode_util import TORCH, U, half_step

COEFFICIENTS = (3.4445, -4.7750, 2.0315)


# ---------------------------------------------------------------- 8 bits

def quantise(X):
    """(Q, scale) by the definition.  127 x and amax have at most 31 and 24 bits, so a quotient that is no tie
    is further from one than 2^-34, and one in 64 bits rounds as the exact one does."""
    x = X.double()
    finite = torch.isfinite(x).all(1, keepdim=True)
    amax = torch.where(finite, x.abs().amax(1, keepdim=True) if x.shape[1] else torch.zeros_like(x.sum(1, keepdim=True)),
                       torch.full((x.shape[0], 1), math.nan, dtype=torch.float64))
    q = torch.where(finite & (amax > 0), torch.round(127 * x / amax), torch.zeros_like(x))
    return q.to(torch.int8), (amax / 127).float()[:, 0]


def int8_product(q, sa, W, sb, bias, dt):
    """(Y, tolerance): conversion of the sum, two factors, the bias: 4 roundings, one to T.  (Products of scales
    below fp32's normal range lose up to half its smallest step before the last factor.)"""
    y = (q.double() @ W.double().t()) * sa.double()[:, None] * sb.double()[None, :]
    b = bias.double()[None, :] if bias is not None else torch.zeros_like(y)
    tol = 4 * U * (y.abs() + b.abs()) + 2.0 ** -149 * (1 + sb.double().abs()[None, :])
    return y + b, tol + half_step(dt, (y + b).abs() + tol)


# ---------------------------------------------------------------- router

def _softmax(x):
    """p, lse and their parts; a row of nothing but -inf: 0."""
    empty = (x == -math.inf).all(1, keepdim=True)
    m = torch.where(empty, torch.zeros((), dtype=torch.float64), x.amax(1, keepdim=True))
    e = torch.exp(x - m)
    s = e.sum(1, keepdim=True)
    p = torch.where(empty, torch.zeros_like(e), e / s)
    lse = torch.where(empty, torch.zeros_like(s), m + torch.log(s))
    bad = (x.isnan() | (x == math.inf)).any(1, keepdim=True)
    nan = torch.full((), math.nan, dtype=torch.float64)
    # |x - max| counts where the exponential is not 0 (2^-150 and below)
    span = torch.where(torch.isfinite(x), (x - m).abs(), torch.zeros_like(x)).clamp(max=104)
    size = torch.where(empty, torch.zeros_like(s), m.abs() + torch.log(s).abs())
    return torch.where(bad, nan, p), torch.where(bad, nan, lse)[:, 0], span, size[:, 0]


def balance(logits, ids, mask):
    """(losses, counts, tokens) and the losses' tolerances."""
    x = logits.double()
    M, E = x.shape
    keep = torch.ones((M,), dtype=torch.bool) if mask is None else mask != 0
    chosen = ids.long()[keep].reshape(-1)
    chosen = chosen[(chosen >= 0) & (chosen < E)]
    counts = torch.bincount(chosen, minlength=E)
    n, total = int(keep.sum()), int(counts.sum())
    p, lse, span, size = _softmax(x)
    p, lse, span, size = p[keep], lse[keep], span[keep], size[keep]
    f = counts.double() / max(total, 1)
    first = E * (f * p.sum(0)).sum() / max(n, 1) if total and n else torch.zeros((), dtype=torch.float64)
    second = (lse * lse).sum() / max(n, 1)
    # a term of p: x - max (|x - max| U), the exponential (2), the sum (E), the quotient (3); the sums over the
    # tokens of one lane (at least 64 workgroups of 16 tokens) and of a workgroup; the rest in 64 bits
    steps = M / 1024 + 24
    ep = E * (f * (p * U * (span + E + 8 + steps)).nan_to_num(0.0).sum(0)).sum() / max(n, 1)
    el = U * (size * 4 + E + 8)
    ez = (2 * lse.abs() * el + lse * lse * U * (steps + 4)).nan_to_num(0.0).sum() / max(n, 1)
    return (torch.stack([first, second]), counts, n), torch.stack([ep + U * first.abs().nan_to_num(0.0),
                                                                   ez + U * second.abs().nan_to_num(0.0)])


def route_grad(logits, ids, g, renorm, mask, counts, n, gl, dt):
    """(gradient, tolerance) from the formula; g or gl may be None."""
    x = logits.double()
    M, E = x.shape
    p, lse, span, size = _softmax(x)
    keep = torch.ones((M,), dtype=torch.bool) if mask is None else mask != 0
    d, s = torch.zeros_like(x), torch.zeros_like(x)  # (s: the terms' sizes)
    if gl is not None and n > 0:
        f = counts.double() / max(int(counts.sum()), 1)
        cb, cz = float(gl[0]) * E / n if int(counts.sum()) else 0.0, float(gl[1]) * 2 / n
        d += cb * p * (f - (p * f).sum(1, keepdim=True)) + cz * lse[:, None] * p
        s += abs(cb) * p * (f + (p * f).sum(1, keepdim=True)) + abs(cz) * p * (size[:, None] + 1)
    if g is not None:
        G, c, Ga = torch.zeros_like(x), torch.zeros_like(x), torch.zeros_like(x)
        for m in range(M):
            for k in range(ids.shape[1]):
                e = int(ids[m, k])
                if 0 <= e < E:
                    G[m, e] += float(g[m, k])
                    Ga[m, e] += abs(float(g[m, k]))
                    c[m, e] += 1
        if renorm:
            D = (p * c).sum(1, keepdim=True)
            r = torch.where(D == 0, torch.zeros_like(D), 1 / D)
            d += p * r * (G - c * (p * G).sum(1, keepdim=True) * r)
            s += p * r * (Ga + c * (p * Ga).sum(1, keepdim=True) * r)
        else:
            d += p * (G - (p * G).sum(1, keepdim=True))
            s += p * (Ga + (p * Ga).sum(1, keepdim=True))
    d[~keep], s[~keep] = 0.0, 0.0
    # p (as above) enters up to three times, through sums over E
    tol = U * s.nan_to_num(0.0) * (3 * (span.amax(1, keepdim=True) + E + 8) + 2 * E + 32) + 1e-37
    return d, tol + half_step(dt, d.abs().nan_to_num(0.0) + tol)


# ---------------------------------------------------------------- orthogonalisation

def orthogonalise(G, steps, dtype=torch.float64):
    """The steps in `dtype`, one matrix."""
    a, b, c = COEFFICIENTS
    X = G.double()
    if not torch.isfinite(X).all():
        return torch.full_like(X, math.nan)
    norm = torch.linalg.vector_norm(X)
    X = (X / norm if float(norm) > 0 else X).to(dtype)
    tall = X.shape[0] > X.shape[1]
    for _ in range(steps):
        A = X.t() @ X if tall else X @ X.t()
        B = b * A + c * (A @ A)
        X = a * X + (X @ B if tall else B @ X)
    return X.double()


def _scalar_bound(x, steps):
    """How far the steps may take one singular value x from its path, in units of e = 2^-22, which is what two
    parts, or a product without lo lo, are off: A = x x is off by 2 e A, A A by 5 e A A, B = a + b A + c A A by
    2 e |b| A + 5 e |c| A A + e |B|, and x' = B x by x times that plus 2 e |B x|, on top of |p'(x)| times what x
    is off (to first order; one unit at the start)."""
    a, b, c = COEFFICIENTS
    off = torch.ones_like(x)
    for _ in range(steps):
        A = x * x
        B = a + b * A + c * A * A
        slope = (a + 3 * b * A + 5 * c * A * A).abs()
        off = slope * off + x.abs() * (2 * abs(b) * A + 5 * abs(c) * A * A + 3 * B.abs())
        x = B * x
    return off


def orthogonalise_tol(G, want, steps, dt):
    """The operands of a product are held to 22 bits where fp32 holds 24, so a rounding is up to 4 times one of
    the same steps in fp32, and the sums are alike.  Those steps' largest error, taken 4 times, twice over as
    either one is a sample; and the rounding to T.

    Where every row and column holds one value, or there is one row or column, the steps in fp32 are paths of
    scalars, which may meet next to no error; their bound is counted instead (_scalar_bound)."""
    nz = G != 0
    if min(G.shape) == 1 or (int(nz.sum(0).max()) <= 1 and int(nz.sum(1).max()) <= 1):
        X = G.double() / torch.linalg.vector_norm(G.double())
        tol = 2.0 ** -22 * (_scalar_bound(X.abs(), steps) if min(G.shape) > 1
                            else _scalar_bound(torch.ones_like(X), steps))
    else:
        worst = 0.0
        for H in (G, -G.flip(0), G.flip(1)):  # (other orders of the same sums)
            e = orthogonalise(H, steps, torch.float32) - orthogonalise(H, steps)
            worst = max(worst, float(e.abs().max()))
        tol = torch.full_like(want, 8 * worst + 2.0 ** -22 * float(want.abs().max()))
    return tol + half_step(dt, want.abs() + tol)


__all__ = ["TORCH", "U", "balance", "half_step", "int8_product", "orthogonalise", "orthogonalise_tol", "quantise",
           "route_grad"]
