"""Plain 64-bit forms of the decode-side operators and the error bounds their
GPU tests use.  Everything here runs on the CPU in torch float64.

Bounds count roundings: u = 2^-24 for an fp32 operation, eps(T) / 2 for a
rounding to T; a sum of n fp32 terms in any order is off by at most n u times
the sum of their magnitudes (the products of 16-bit values are exact in fp32).
"""
import math

import torch

U = 2.0 ** -24
TORCH = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
# two halves of T hold an fp32 value to this relative error (fp32 itself: exact)
SPLIT = {"bf16": 2.0 ** -16, "f16": 2.0 ** -20, "f32": 0.0}


def half_step(dt, y):
    """Half a step of T at |y|, with the smallest subnormal's half as a floor."""
    fi = torch.finfo(TORCH[dt])
    return fi.eps / 2 * y.abs() + fi.smallest_normal * fi.eps


def draw(gen, shape, std, dt):
    return (torch.randn(shape, generator=gen) * std).to(TORCH[dt])


def assert_within(got, want, tol, what=""):
    got, want = got.double().cpu(), want.double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    same = (got == want) | (got.isnan() & want.isnan())
    bad = ~(same | ((got - want).abs() <= tol))
    if bad.any():
        i = int(torch.where(bad, (got - want).abs() / tol, torch.zeros_like(want)).nan_to_num(nan=1e300).argmax())
        raise AssertionError("%s: %d / %d outside; worst at %d: got %r want %r tol %r" % (
            what, int(bad.sum()), bad.numel(), i, float(got.flatten()[i]), float(want.flatten()[i]),
            float(tol.flatten()[i]) if torch.is_tensor(tol) else tol))


# ---------------------------------------------------------------- adapters

def lora(X, W, A, B, idx, scale, bias, trans, dt):
    """(Y, tolerance)."""
    X, W, A, B = (t.double() for t in (X, W, A, B))
    if trans:
        W, A, B = W.t(), A.transpose(1, 2), B.transpose(1, 2)
    K, R = X.shape[1], A.shape[2]
    Y, S = X @ W, X.abs() @ W.abs()
    D, SD = torch.zeros_like(Y), torch.zeros_like(Y)
    if bias is not None:
        D, SD = D + bias.double(), SD + bias.double().abs()
    for m, g in enumerate(idx.tolist()):
        if 0 <= g < A.shape[0]:
            s = float(scale[g]) if scale is not None else 1.0
            D[m] += s * ((X[m] @ A[g]) @ B[g])
            SD[m] += abs(s) * ((X[m].abs() @ A[g].abs()) @ B[g].abs())
    # sums over K and R, the scale, the joins; the adapter's middle value may be held in two halves of T
    tol = (K + 8) * U * S + ((K + R + 16) * U + SPLIT[dt]) * SD
    # one rounding of the sum; long batches and element-wise layouts also round the adapter's term
    return Y + D, tol + half_step(dt, D) + half_step(dt, (Y + D).abs() + tol)


# ---------------------------------------------------------------- router

def route(logits, k, renorm):
    x = logits.double()
    # NaN first, then by value; a stable sort leaves ties in index order
    key = torch.where(x.isnan(), torch.full_like(x, math.inf), x)
    order = torch.argsort(key, dim=1, descending=True, stable=True)
    nan = x.isnan().gather(1, order)
    order = order.gather(1, torch.argsort(nan.to(torch.int8), dim=1, descending=True, stable=True))
    ids = order[:, :k]
    p = torch.softmax(x, 1)
    p = torch.where((x == -math.inf).all(1, keepdim=True), torch.zeros_like(p), p)
    w = p.gather(1, ids)
    if renorm:
        s = w.sum(1, keepdim=True)
        w = torch.where(s == 0, torch.zeros_like(w), w / s)
    return ids, w


def route_tol(logits, ids, w):
    """Weights: e^(x - max) with |x - max| rounded once, a sum of up to E terms, a division."""
    x = logits.double()
    span = (x.amax(1, keepdim=True) - x.gather(1, ids)).abs().clamp(max=120)
    return w * U * (span + x.shape[1] + 8) + 1e-37


# ---------------------------------------------------------------- expert layer

def act(x, name):
    return x * torch.sigmoid(x) if name == "silu" else 0.5 * x * (1 + torch.erf(x / math.sqrt(2.0)))


def moe(X, logits, k, Wg, Wu, Wd, renorm, activation, trans, dt):
    """(Y, tolerance)."""
    ids, w = route(logits, k, renorm)
    dw = route_tol(logits, ids, w)
    X = X.double()
    K = X.shape[1]
    Y, tol = torch.zeros_like(X), torch.zeros_like(X)
    for e in ids.unique().tolist():
        rows, slots = torch.nonzero(ids == e, as_tuple=True)
        g_, u_, d_ = (t[e].double().t() if trans else t[e].double() for t in (Wg, Wu, Wd))
        F = g_.shape[1]
        x = X[rows]
        g, u = x @ g_, x @ u_
        eg, eu = (K + 8) * U * (x.abs() @ g_.abs()), (K + 8) * U * (x.abs() @ u_.abs())
        a = act(g, activation)
        # |act'| <= 1.13; act itself a few fp32 operations, e^-x and erf within 4 u of the branch's size
        ea = 1.13 * eg + 16 * U * (a.abs() + g.abs() * 0.5)
        ww, ew = w[rows, slots][:, None], dw[rows, slots][:, None]
        h = a * u * ww
        eh = ea * u.abs() * ww + (a.abs() + ea) * eu * ww + a.abs() * u.abs() * ew + (4 * U + SPLIT[dt]) * h.abs()
        Y[rows] += h @ d_
        tol[rows] += eh @ d_.abs() + (k * F + 16) * U * (h.abs() @ d_.abs())
    return Y, tol + half_step(dt, Y.abs() + tol)


# ---------------------------------------------------------------- log probabilities

def logprobs(logits, targets, k):
    """(logprobs, entropy, lse, ids, top logprobs) and their tolerances (ids: None)."""
    x = logits.double()
    M, V = x.shape
    m = x.amax(1, keepdim=True)
    empty = (x == -math.inf).all(1, keepdim=True)
    m0 = torch.where(empty, torch.zeros_like(m), m)
    d = x - m0
    e = torch.exp(d)
    s = e.sum(1, keepdim=True)
    logs = torch.log(s)
    lse = torch.where(empty, torch.full_like(m, -math.inf), m0 + logs)
    lp = torch.where(empty, torch.full_like(x, -math.inf), d - logs)
    p = torch.where(empty, torch.zeros_like(e), e / s)
    bad = (x.isnan() | (x == math.inf)).any(1, keepdim=True)
    lp = torch.where(bad, torch.full_like(lp, math.nan), lp)
    ent = torch.where(empty | (p == 0).all(1, keepdim=True), torch.zeros_like(logs),
                      -(p * torch.where(p > 0, lp, torch.zeros_like(lp))).sum(1, keepdim=True))
    ent = torch.where(bad, torch.full_like(ent, math.nan), ent)
    lse = torch.where(bad, torch.full_like(lse, math.nan), lse)
    ids, _ = route(logits, k, False) if k else (torch.zeros((M, 0), dtype=torch.int64), None)
    t = targets.to(torch.int64)
    valid = (t >= 0) & (t < V)
    lpt = torch.where(valid, lp.gather(1, t.clamp(0, V - 1)[:, None])[:, 0], torch.zeros((M,), dtype=torch.float64))
    # roundings of a term e^(x - m): x - m, its product with log2 e, the exponential (1 ulp): u (3 |d| + 2);
    # every maximum passed on the way rescales by such a term (the steps of d add up to the row's span);
    # adds: V in the worst order, counted for the terms' mean as the sums' magnitudes are the sums themselves
    # (e^-120 and below are 0 in fp32: no error)
    fin = torch.where(torch.isfinite(d), d, torch.zeros_like(d)).abs()
    near = fin.clamp(max=120)
    span = near.amax(1, keepdim=True)
    ed = (p * near).sum(1, keepdim=True)
    ed2 = (p * near * near).sum(1, keepdim=True)
    n = V / 256 + 64
    es = U * (3 * ed + 3 * span + 3 * n)
    et = U * (3 * ed2 + (3 * span + 3 * n + 4) * ed + ed * n)
    ln = logs.abs()
    tol_lp = es + U * (fin + 3 * ln + lp.nan_to_num(0, 0, 0).abs() + 4)
    tol_lse = (es + U * (4 * ln + m0.abs() + (m0 + logs).abs() + 4))[:, 0]
    tol_ent = (es + et + es * ed + U * (4 * ln + 4 * ed + 8))[:, 0]
    tol_t = tol_lp.gather(1, t.clamp(0, V - 1)[:, None])[:, 0]
    return (lpt, ent[:, 0], lse[:, 0], ids, lp.gather(1, ids)), (tol_t, tol_ent, tol_lse, None, tol_lp.gather(1, ids))


def logprobs_grad(logits, targets, lse, gl, entropy, gh, dt):
    """(gradient, tolerance) from the formula, with lse and entropy as given."""
    x, lse = logits.double(), lse.double()[:, None]
    M, V = x.shape
    t = targets.to(torch.int64)
    valid = (t >= 0) & (t < V)
    gl = (gl.double() * valid)[:, None]
    empty = lse == -math.inf
    l = torch.where(empty, torch.full_like(x, -math.inf), x - torch.where(empty, torch.zeros_like(lse), lse))
    p = torch.exp(l)
    lf = torch.where(p == 0, torch.zeros_like(l), l)
    hot = torch.zeros_like(x)
    hot[torch.arange(M)[valid], t[valid]] = 1.0
    hot = torch.where(empty, torch.zeros_like(hot), hot)
    g = gl * (hot - p)
    size = gl.abs() * (hot + p)
    if gh is not None:
        H, gh = entropy.double()[:, None], gh.double()[:, None]
        g = g - gh * p * (lf + H)
        size = size + gh.abs() * p * (lf.abs() + H.abs())
    tol = U * size * (3 * lf.abs() + 8) + 1e-37
    return g, tol + half_step(dt, g.abs() + tol)
