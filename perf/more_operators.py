"""The measured cases of the operators that train, balance and quantise the
weights of the products: 8-bit products with a scale for each token and channel,
the router's balance loss and gradient, and the orthogonalised weight update.

Each operator is written twice: in its plain form (elementary torch operations
in 32 bits, rounded once at the end) and as the calls a program makes of this
package (`own` true).  `exact` holds the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
# Newton-Schulz steps X <- a X + (b A + c A^2) X, A = X X^T
COEFFICIENTS = (3.4445, -4.7750, 2.0315)


# ---------------------------------------------------------------------------- cases

def _linear(dtype, M, K, N, bias):
    """A projection whose input is quantised by the call: W (N, K) in int8, a scale for each of its rows."""
    return dict(op="linear", dtype=dtype, M=M, K=K, N=N, bias=bias)


def _shared(dtype, M, K, N, share):
    """Three projections of one input, quantised once: N columns, and twice N / share (grouped heads)."""
    return dict(op="shared", dtype=dtype, M=M, K=K, N=N, share=share)


def _balance(dtype, M, E, top_k, padded):
    """padded: the share of tokens that a mask leaves out."""
    return dict(op="balance", dtype=dtype, M=M, E=E, top_k=top_k, padded=padded)


def _route_grad(dtype, M, E, top_k, renormalize, padded):
    return dict(op="route_grad", dtype=dtype, M=M, E=E, top_k=top_k, renormalize=renormalize, padded=padded)


def _orthogonal(dtype, batch, rows, cols, rank):
    """rank: of the part that stands out of the update's noise."""
    return dict(op="orthogonal", dtype=dtype, batch=batch, rows=rows, cols=cols, rank=rank)


def listed():
    cases = [
        # one request's next token through a square projection
        ("linear_1", _linear("bf16", 1, 4096, 4096, False)),
        # a decode batch; rows and width are odd
        ("linear_43", _linear("f16", 43, 4096, 4104, True)),
        # prompts of several requests in one call
        ("linear_8192", _linear("bf16", 8192, 4096, 8192, False)),
        # a short prompt through query, key and value projections; the contraction is odd, so rows are not aligned
        ("shared_300", _shared("f16", 300, 2005, 2048, 4)),
        # a prompt batch through the same of a wide model with few key and value heads
        ("shared_4096", _shared("bf16", 4096, 8192, 1024, 8)),
        # a training batch's router, at the grouped product's benchmark size
        ("balance_16384", _balance("bf16", 16384, 64, 8, 0.0)),
        # a padded batch in fp32 over an odd number of experts
        ("balance_1000", _balance("f32", 1000, 60, 4, 0.3)),
        # the gradients of those two
        ("route_grad_16384", _route_grad("bf16", 16384, 64, 8, True, 0.0)),
        ("route_grad_1000", _route_grad("f32", 1000, 60, 4, False, 0.3)),
        # the update of one projection of a small model, kept in fp32
        ("orthogonal_512", _orthogonal("f32", 1, 512, 1024, 16)),
        # the down projections of an expert layer, taller than wide; the width is odd
        ("orthogonal_experts", _orthogonal("bf16", 16, 1024, 1000, 16)),
        # a square projection
        ("orthogonal_4096", _orthogonal("bf16", 1, 4096, 4096, 64)),
    ]
    return [dict(case, name=name) for name, case in cases]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi, step):
    """A size spread over the logarithm; three in four are multiples of `step`, the rest are as drawn."""
    n = _log_int(rng, lo, hi)
    return max(step, n // step * step) if rng.random() < 0.75 else n


def draw(rng):
    op = rng.choice(["linear", "linear", "shared", "balance", "route_grad", "orthogonal"])
    half = rng.choice(["bf16", "bf16", "f16"])
    if op in ("linear", "shared"):
        dtype = half if rng.random() < 0.9 else "f32"
        M = _log_int(rng, 1, 64) if rng.random() < 0.5 else _log_int(rng, 65, 8192)
        if op == "linear":
            return _linear(dtype, M, _width(rng, 256, 4096, 64), _width(rng, 256, 8192, 64), rng.random() < 0.5)
        return _shared(dtype, min(M, 4096), _width(rng, 512, 8192, 64), _width(rng, 512, 2048, 64),
                       rng.choice([1, 2, 4, 8]))
    if op in ("balance", "route_grad"):
        E = rng.choice([8, 16, 60, 64, 128, 160, 256])
        dtype, M, k = rng.choice(["f32", "bf16", "f16"]), _log_int(rng, 16, 65536), rng.randint(1, min(8, E))
        padded = rng.choice([0.0, 0.3])
        return (_balance(dtype, M, E, k, padded) if op == "balance" else
                _route_grad(dtype, M, E, k, rng.random() < 0.5, padded))
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    rows, cols = _width(rng, 64, 4096, 64), _width(rng, 64, 4096, 64)
    room = 4096 ** 3 // (rows * cols * min(rows, cols))
    batch = 1 if rng.random() < 0.5 else _log_int(rng, 1, max(1, min(32, room)))
    return _orthogonal(dtype, batch, rows, cols, rng.choice([0, 4, 16, 64]))


def _projections(case):
    """Widths of the projections of a "linear" or "shared" case."""
    N = case["N"]
    return [N] if case["op"] == "linear" else [N] + [max(1, N // case["share"])] * 2


def work(case):
    op, b = case["op"], BYTES[case["dtype"]]
    if op in ("linear", "shared"):
        M, K, N = case["M"], case["K"], sum(_projections(case))
        return {"bytes": M * K * b + N * K + M * N * b, "flops": 2 * M * K * N}
    if op in ("balance", "route_grad"):
        M, E, k = case["M"], case["E"], case["top_k"]
        if op == "balance":
            return {"bytes": M * E * b + M * k * 4, "flops": 6 * M * E}
        return {"bytes": 2 * M * E * b + M * k * 8, "flops": 12 * M * E}
    lo, hi = sorted((case["rows"], case["cols"]))
    # 5 steps: the two symmetric products by half, the third whole
    return {"bytes": 2 * case["batch"] * lo * hi * b, "flops": 5 * case["batch"] * (3 * lo * lo * hi + lo ** 3)}


# ---------------------------------------------------------------------------- inputs

def _normal(gen, shape, std, dtype):
    """N(0, std) of `dtype`, drawn in it (the draws of a large tensor need no fp32 copy)."""
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def _quantised_weights(gen, N, K):
    """A trained projection's rows in int8, each with a scale of its own."""
    W = torch.empty((N, K), device="cuda").normal_(0.0, K ** -0.5, generator=gen)
    W *= torch.rand((N, 1), generator=gen, device="cuda") + 0.5
    scale = W.abs().amax(1) / 127
    return torch.round(W / scale[:, None]).clamp(-127, 127).to(torch.int8), scale


def _router(st, gen, case):
    M, E, k = case["M"], case["E"], case["top_k"]
    # some experts are liked more than others
    x = torch.empty((M, E), device="cuda").normal_(0.0, 1.5, generator=gen)
    x += torch.empty((1, E), device="cuda").normal_(0.0, 0.7, generator=gen)
    st["logits"] = x.to(DTYPES[case["dtype"]])
    st["indices"] = torch.topk(st["logits"].float(), k, dim=1)[1].to(torch.int32)
    st["mask"] = torch.rand((M,), generator=gen, device="cuda") >= case["padded"] if case["padded"] else None


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt, op = DTYPES[case["dtype"]], case["op"]
    st = dict(case=case)
    if op in ("linear", "shared"):
        M, K = case["M"], case["K"]
        X = torch.empty((M, K), device="cuda").normal_(0.0, 1.0, generator=gen)
        # tokens of different sizes, and some channels that stand out
        X *= torch.rand((M, 1), generator=gen, device="cuda") * 2 + 0.2
        X *= 1 + 7 * (torch.rand((1, K), generator=gen, device="cuda") < 0.01)
        st["X"] = X.to(dt)
        st["W"] = [_quantised_weights(gen, n, K) for n in _projections(case)]
        st["bias"] = _normal(gen, (case["N"],), 0.1, dt) if case.get("bias") else None
    elif op in ("balance", "route_grad"):
        _router(st, gen, case)
        if op == "route_grad":
            M, E = case["M"], case["E"]
            # what the forward pass has left behind
            keep = st["mask"] if st["mask"] is not None else torch.ones((M,), dtype=torch.bool, device="cuda")
            chosen = st["indices"][keep].to(torch.int64).reshape(-1)
            st["counts"] = torch.bincount(chosen, minlength=E).to(torch.int32)
            st["tokens"] = keep.sum().to(torch.int32).reshape(1)
            # of a loss summed over the tokens
            st["g_weights"] = torch.randn((M, case["top_k"]), generator=gen, device="cuda")
            st["g_losses"] = torch.tensor([0.01 * M, 0.001 * M], device="cuda")
    else:
        B, m, n, r = case["batch"], case["rows"], case["cols"], case["rank"]
        shape = (m, n) if B == 1 else (B, m, n)
        # a momentum: noise, and a few directions well above it
        G = torch.empty((B, m, n), device="cuda").normal_(0.0, 1e-3, generator=gen)
        if r:
            U = torch.empty((B, m, r), device="cuda").normal_(0.0, 1e-3, generator=gen)
            U *= torch.linspace(1.0, 0.1, r, device="cuda")
            G += U @ torch.empty((B, r, n), device="cuda").normal_(0.0, 1.0, generator=gen)
        st["G"] = G.reshape(shape).to(dt)
    return st


# ---------------------------------------------------------------------------- plain forms

def _plain_quantise(X):
    # in 64 bits: a value next to the border of two steps goes to the nearer one
    x = X.double()
    scale = x.abs().amax(1, keepdim=True) / 127
    q = torch.round(x / torch.where(scale > 0, scale, torch.ones_like(scale)))
    return q.float(), scale.float()


def _plain_product(q, scale, W, w_scale, bias, dt):
    y = (q @ W.float().t()) * scale * w_scale[None, :]
    if bias is not None:
        y = y + bias.float()
    return y.to(dt)


def _softmax(x):
    m = x.amax(1, keepdim=True)
    e = torch.exp(x - m)
    s = e.sum(1, keepdim=True)
    return e / s, (m + torch.log(s))[:, 0]


def _plain_balance(st):
    x, ids = st["logits"].float(), st["indices"].to(torch.int64)
    M, E = x.shape
    keep = torch.ones((M,), device=x.device) if st["mask"] is None else st["mask"].float()
    p, lse = _softmax(x)
    n = keep.sum()
    counts = torch.zeros((E,), device=x.device).scatter_add_(0, ids.reshape(-1), keep[:, None].expand_as(ids).reshape(-1))
    balance = E * (counts / counts.sum() * (p * keep[:, None]).sum(0)).sum() / n
    z = (keep * lse * lse).sum() / n
    return torch.stack([balance, z]), counts.to(torch.int32), n.to(torch.int32).reshape(1)


def _plain_route_grad(st):
    x, ids, g = st["logits"].float(), st["indices"].to(torch.int64), st["g_weights"]
    p, lse = _softmax(x)
    n, c = st["tokens"].float(), st["counts"].float()
    E = x.shape[1]
    f = c / c.sum()
    d = (st["g_losses"][0] * E / n) * p * (f[None, :] - (p * f[None, :]).sum(1, keepdim=True))
    d = d + (st["g_losses"][1] * 2 / n) * lse[:, None] * p
    w = p.gather(1, ids)
    if st["case"]["renormalize"]:
        w = w / w.sum(1, keepdim=True)
        d = d.scatter_add(1, ids, w * (g - (w * g).sum(1, keepdim=True)))
    else:
        d = d - p * (w * g).sum(1, keepdim=True)
        d = d.scatter_add(1, ids, w * g)
    if st["mask"] is not None:
        d = d * st["mask"].float()[:, None]
    return d.to(st["logits"].dtype)


def _plain_orthogonal(st):
    G = st["G"]
    X = G.float()
    tall = X.shape[-2] > X.shape[-1]
    if tall:
        X = X.transpose(-1, -2).contiguous()
    X = X / X.square().sum((-1, -2), keepdim=True).sqrt()
    a, b, c = COEFFICIENTS
    for _ in range(5):
        A = X @ X.transpose(-1, -2)
        X = a * X + (b * A + c * (A @ A)) @ X
    if tall:
        X = X.transpose(-1, -2).contiguous()
    return X.to(G.dtype)


def _plain(st):
    op = st["case"]["op"]
    if op in ("linear", "shared"):
        q, scale = _plain_quantise(st["X"])
        return [_plain_product(q, scale, W, s, st["bias"], st["X"].dtype) for W, s in st["W"]]
    if op == "balance":
        return _plain_balance(st)
    if op == "route_grad":
        return _plain_route_grad(st)
    return _plain_orthogonal(st)


# ---------------------------------------------------------------------------- one pass

def run(st):
    if not own:
        return _plain(st)
    import onnx_matmul_family_amd as omm
    case = st["case"]
    if case["op"] == "linear":
        W, s = st["W"][0]
        return [omm.int8_matmul(st["X"], W, s, bias=st["bias"])[0]]
    if case["op"] == "shared":
        q, scale = omm.quantize_rows(st["X"])
        return [omm.int8_matmul(q, W, s, a_scale=scale, dtype=st["X"].dtype)[0] for W, s in st["W"]]
    if case["op"] == "balance":
        return omm.moe_balance(st["logits"], st["indices"], token_mask=st["mask"])
    if case["op"] == "route_grad":
        return omm.moe_route_grad(st["logits"], st["indices"], st["g_weights"], renormalize=case["renormalize"],
                                  token_mask=st["mask"], counts=st["counts"], tokens=st["tokens"],
                                  grad_losses=st["g_losses"])
    return omm.orthogonalize(st["G"])[0]


# ---------------------------------------------------------------------------- definitions in 64 bits

def _exact_linear(st):
    out = []
    x = st["X"].double()
    big = x.abs().max(dim=1, keepdim=True)[0]
    q = torch.where(big > 0, torch.round(x * 127 / big.clamp(min=1e-300)), torch.zeros_like(x))
    for W, s in st["W"]:
        y = torch.mm(q, W.double().t().contiguous())
        y = y * (big / 127) * s.double()
        out.append(y if st["bias"] is None else y + st["bias"].double())
    return out


def _losses(x, ids, keep, counts):
    """(balance, z) of the counted tokens; x in 64 bits."""
    logp = torch.log_softmax(x[keep], 1)
    mean = logp.exp().mean(0)
    share = counts.double() / counts.double().sum()
    lse = torch.logsumexp(x[keep], 1)
    return torch.stack([x.shape[1] * torch.dot(share, mean), lse.square().mean()])


def _keep(st):
    if st["mask"] is not None:
        return st["mask"]
    return torch.ones((st["logits"].shape[0],), dtype=torch.bool, device="cuda")


def _exact_balance(st):
    x, keep = st["logits"].double(), _keep(st)
    counts = torch.bincount(st["indices"][keep].to(torch.int64).reshape(-1), minlength=x.shape[1])
    return (_losses(x, st["indices"], keep, counts), counts.to(torch.int32),
            torch.count_nonzero(keep).to(torch.int32).reshape(1))


def _exact_route_grad(st):
    # the gradient of the formula itself
    x = st["logits"].double().requires_grad_(True)
    keep, ids = _keep(st), st["indices"].to(torch.int64)
    if st["case"]["renormalize"]:
        w = torch.softmax(x.gather(1, ids), 1)
    else:
        w = torch.softmax(x, 1).gather(1, ids)
    total = (w * st["g_weights"].double())[keep].sum()
    total = total + torch.dot(_losses(x, ids, keep, st["counts"]), st["g_losses"].double())
    return torch.autograd.grad(total, x)[0]


def _exact_orthogonal(st):
    G = st["G"].double()
    G = G if G.dim() == 3 else G[None]
    out = []
    for X in G:
        X = X / torch.linalg.vector_norm(X)
        wide = X.shape[0] < X.shape[1]
        for _ in range(5):
            # an odd polynomial of X: the products may stand on either side; here on the shorter one,
            # with X (X^T X) in steps
            a, b, c = COEFFICIENTS
            Xt = X.t().contiguous()
            if wide:
                Y = torch.mm(torch.mm(X, Xt), X)
                X = a * X + b * Y + c * torch.mm(torch.mm(X, Xt), Y)
            else:
                Y = torch.mm(X, torch.mm(Xt, X))
                X = a * X + b * Y + c * torch.mm(Y, torch.mm(Xt, X))
        out.append(X)
    return torch.stack(out).reshape(st["G"].shape)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("linear", "shared"):
        return _exact_linear(st)
    if case["op"] == "balance":
        return _exact_balance(st)
    if case["op"] == "route_grad":
        return _exact_route_grad(st)
    return _exact_orthogonal(st)
