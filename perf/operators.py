"""The measured cases of the decode-side operators: a projection with low-rank
adapters, the expert router, the expert layer of a few tokens, and the log
probabilities of given tokens with their gradient.

Each operator is written twice: in its plain form (elementary torch operations
in 32 bits, rounded once at the end) and as the calls a program makes of this
package (`own` true).  `exact` holds the definitions in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


# ---------------------------------------------------------------------------- cases

def _lora(dtype, M, K, N, R, G, trans, rows, bias):
    """rows: "mixed" = every row its own request (decode), "runs" = requests of many rows (prompts)."""
    return dict(op="lora", dtype=dtype, M=M, K=K, N=N, R=R, G=G, trans=trans, rows=rows, bias=bias)


def _route(dtype, M, E, top_k, renormalize):
    return dict(op="route", dtype=dtype, M=M, E=E, top_k=top_k, renormalize=renormalize)


def _moe(dtype, M, K, F, E, top_k, trans, renormalize, activation):
    return dict(op="moe", dtype=dtype, M=M, K=K, F=F, E=E, top_k=top_k, trans=trans, renormalize=renormalize,
                activation=activation)


def _logprobs(dtype, M, V, top_k, masked):
    """masked: the share of the vocabulary that a grammar or filter has set to -inf."""
    return dict(op="logprobs", dtype=dtype, M=M, V=V, top_k=top_k, masked=masked)


def _logprobs_grad(dtype, M, V, entropy, ignored):
    """ignored: the share of rows whose target is -1 (prompt or padding)."""
    return dict(op="logprobs_grad", dtype=dtype, M=M, V=V, entropy=entropy, ignored=ignored)


def listed():
    cases = [
        # one request's next token through a square projection
        ("lora_decode_1", _lora("bf16", 1, 4096, 4096, 16, 8, True, "mixed", False)),
        # a decode batch in which most requests bring an adapter of their own; rows, width and rank are odd
        ("lora_decode_43", _lora("f16", 43, 4096, 4104, 24, 32, False, "mixed", True)),
        # several prompts of different adapters in one call
        ("lora_prompts", _lora("bf16", 4096, 4096, 8192, 32, 8, True, "runs", False)),
        # the router of one token
        ("route_1", _route("f32", 1, 64, 8, True)),
        # the router of a whole prompt batch, at the grouped product's benchmark size
        ("route_16384", _route("bf16", 16384, 64, 8, False)),
        # one token through the grouped product's benchmark experts
        ("moe_1", _moe("bf16", 1, 4096, 2048, 64, 8, False, True, "silu")),
        # a small decode batch over small experts stored as linear layers store them; the width is odd
        ("moe_23_small", _moe("f16", 23, 1024, 1000, 16, 4, True, False, "gelu")),
        # a decode batch that reaches nearly every expert
        ("moe_32", _moe("bf16", 32, 4096, 2048, 64, 8, False, True, "silu")),
        # one sampled token of a served request with its alternatives, part of the vocabulary masked
        ("logprobs_1", _logprobs("bf16", 1, 131072, 5, 0.25)),
        # scoring a batch of sequences; the vocabulary is odd, so rows are not aligned
        ("logprobs_2048", _logprobs("bf16", 2048, 50001, 20, 0.0)),
        # a small training batch in fp32
        ("logprobs_grad_64", _logprobs_grad("f32", 64, 32000, False, 0.3)),
        # a training batch with an entropy term
        ("logprobs_grad_4096", _logprobs_grad("bf16", 4096, 131072, True, 0.1)),
    ]
    return [dict(case, name=name) for name, case in cases]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi, step):
    """A size spread over the logarithm; three in four are multiples of `step`, the rest are as drawn."""
    n = _log_int(rng, lo, hi)
    return max(step, n // step * step) if rng.random() < 0.75 else n


def draw(rng):
    op = rng.choice(["lora", "route", "moe", "logprobs", "logprobs_grad"])
    half = rng.choice(["bf16", "bf16", "f16"])
    if op == "lora":
        few = rng.random() < 0.6
        dtype = half if rng.random() < 0.9 else "f32"
        M = _log_int(rng, 1, 64) if few else _log_int(rng, 65, 4096 if dtype != "f32" else 512)
        return _lora(dtype, M, _width(rng, 512, 4096, 64), _width(rng, 512, 8192, 64),
                     rng.choice([4, 8, 16, 16, 24, 32, 64]), rng.randint(1, 32), rng.random() < 0.5,
                     "mixed" if few else rng.choice(["runs", "runs", "mixed"]), rng.random() < 0.5)
    if op == "route":
        E = rng.choice([8, 16, 60, 64, 128, 160, 256])
        return _route(rng.choice(["f32", "bf16", "f16"]), _log_int(rng, 1, 16384), E, rng.randint(1, min(8, E)),
                      rng.random() < 0.5)
    if op == "moe":
        E = rng.choice([4, 8, 16, 60, 64])
        dtype = half if rng.random() < 0.9 else "f32"
        return _moe(dtype, _log_int(rng, 1, 32), _width(rng, 256, 4096, 64), _width(rng, 128, 2048, 64), E,
                    rng.randint(1, min(8, E)), rng.random() < 0.5, rng.random() < 0.5, rng.choice(["silu", "gelu"]))
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    M, V = _log_int(rng, 1, 2048), _width(rng, 1000, 131072, 64)
    if op == "logprobs":
        return _logprobs(dtype, M, V, rng.choice([0, 1, 5, 10, 20]), rng.choice([0.0, 0.25, 0.9]))
    return _logprobs_grad(dtype, M, V, rng.random() < 0.5, rng.choice([0.0, 0.3]))


def work(case):
    op, b = case["op"], BYTES[case["dtype"]]
    M = case["M"]
    if op == "lora":
        K, N, R = case["K"], case["N"], case["R"]
        # adapters in use: rows that draw uniformly from G + 1 choices (one of them none)
        G = case["G"]
        used = G * (1 - (1 - 1 / (G + 1)) ** M) if case["rows"] == "mixed" else min(G, M)
        return {"bytes": int(b * (M * K + K * N + M * N + used * R * (K + N))),
                "flops": 2 * M * K * N + 2 * M * R * (K + N)}
    if op == "route":
        return {"bytes": M * case["E"] * b + M * case["top_k"] * 8, "flops": 4 * M * case["E"]}
    if op == "moe":
        K, F, E, S = case["K"], case["F"], case["E"], case["top_k"]
        used = E * (1 - (1 - S / E) ** M)
        return {"bytes": int(b * (2 * M * K + used * 3 * K * F) + b * M * E), "flops": 6 * M * S * K * F}
    V = case["V"]
    if op == "logprobs":
        return {"bytes": M * V * b + M * (16 + 8 * case["top_k"]), "flops": 5 * M * V}
    return {"bytes": 2 * M * V * b + M * 20, "flops": 5 * M * V}


# ---------------------------------------------------------------------------- inputs

def _normal(gen, shape, std, dtype):
    """N(0, std) of `dtype`, drawn in it (the draws of a large tensor need no fp32 copy)."""
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def _logits(gen, M, V, dtype, masked):
    """Next-token logits: a broad spread with a few likely tokens in each row."""
    x = torch.empty((M, V), dtype=torch.float32, device="cuda").normal_(0.0, 2.0, generator=gen)
    likely = torch.randint(0, V, (M, 4), generator=gen, device="cuda")
    x.scatter_add_(1, likely, torch.rand((M, 4), generator=gen, device="cuda") * 8 + 6)
    if masked > 0:
        x.masked_fill_((torch.rand((V,), generator=gen, device="cuda") < masked)[None, :], -math.inf)
    return x.to(dtype), likely


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    op, M = case["op"], case["M"]
    st = dict(case=case)
    if op == "lora":
        K, N, R, G, trans = case["K"], case["N"], case["R"], case["G"], case["trans"]
        st["X"] = _normal(gen, (M, K), 1.0, dt)
        st["W"] = _normal(gen, (N, K) if trans else (K, N), K ** -0.5, dt)
        st["A"] = _normal(gen, (G, R, K) if trans else (G, K, R), K ** -0.5, dt)
        st["B"] = _normal(gen, (G, N, R) if trans else (G, R, N), 0.5 * R ** -0.5, dt)
        st["scale"] = torch.rand((G,), generator=gen, device="cuda") * 1.5 + 0.5
        st["bias"] = _normal(gen, (N,), 0.1, dt) if case["bias"] else None
        idx = torch.randint(-1, G, (M,), generator=gen, device="cuda", dtype=torch.int32)
        if case["rows"] == "runs":  # prompts of uneven length, one adapter (or none) each
            ends = torch.sort(torch.randint(0, M, (G - 1,), generator=gen, device="cuda"))[0]
            run = (torch.arange(M, device="cuda")[:, None] >= ends[None, :]).sum(1)
            idx = ((run + seed) % (G + 1) - 1).to(torch.int32)
        st["idx"] = idx
        if own:
            import onnx_matmul_family_amd as omm
            st["ws"] = torch.empty(omm.lora_matmul_workspace_size(M, K, N, R, dt), dtype=torch.uint8, device="cuda")
    elif op == "route":
        st["logits"] = _normal(gen, (M, case["E"]), 1.5, dt)
    elif op == "moe":
        K, F, E, trans = case["K"], case["F"], case["E"], case["trans"]
        st["X"] = _normal(gen, (M, K), 1.0, dt)
        st["logits"] = _normal(gen, (M, E), 1.5, torch.float32)
        up, down = ((E, F, K), (E, K, F)) if trans else ((E, K, F), (E, F, K))
        st["W_gate"] = _normal(gen, up, K ** -0.5, dt)
        st["W_up"] = _normal(gen, up, K ** -0.5, dt)
        st["W_down"] = _normal(gen, down, F ** -0.5, dt)
        if own:
            import onnx_matmul_family_amd as omm
            st["ws"] = torch.empty(omm.moe_layer_workspace_size(M, K, F, E, case["top_k"]), dtype=torch.uint8,
                                   device="cuda")
    else:
        V = case["V"]
        st["logits"], likely = _logits(gen, M, V, dt, case.get("masked", 0.0))
        st["targets"] = torch.where(torch.rand((M,), generator=gen, device="cuda") < 0.5, likely[:, 0],
                                    torch.randint(0, V, (M,), generator=gen, device="cuda")).to(torch.int64)
        if op == "logprobs_grad":
            drop = torch.rand((M,), generator=gen, device="cuda") < case["ignored"]
            st["targets"] = st["targets"].masked_fill(drop, -1)
            st["g_logprobs"] = torch.randn((M,), generator=gen, device="cuda") * (1.0 / M) ** 0.5
            st["g_entropy"] = (torch.randn((M,), generator=gen, device="cuda") * 0.1 * (1.0 / M) ** 0.5
                               if case["entropy"] else None)
            # what the forward pass has left behind
            lse, ent = [], []
            for x in st["logits"].split(256):
                x = x.double()
                l = torch.logsumexp(x, 1)
                p = torch.exp(x - l[:, None])
                lse.append(l)
                ent.append(l - (p * x).sum(1))
            st["lse"] = torch.cat(lse).float()
            st["entropy"] = torch.cat(ent).float()
        elif own:
            import onnx_matmul_family_amd as omm
            st["ws"] = torch.empty(omm.token_logprobs_workspace_size(M, V, case["top_k"]), dtype=torch.uint8,
                                   device="cuda")
    return st


# ---------------------------------------------------------------------------- plain forms

def _plain_lora(st):
    case = st["case"]
    X, W, A, B = st["X"].float(), st["W"].float(), st["A"], st["B"]
    if case["trans"]:
        W, A, B = W.t(), A.transpose(1, 2), B.transpose(1, 2)
    Y = X @ W
    if st["bias"] is not None:
        Y = Y + st["bias"].float()
    idx, scale = st["idx"], st["scale"]
    if case["M"] <= case["G"]:  # gather each row's adapter
        on = (idx >= 0).float()
        g = idx.clamp(min=0).long()
        T = (X[:, :, None] * A[g].float()).sum(1) * (scale[g] * on)[:, None]
        Y = Y + (T[:, :, None] * B[g].float()).sum(1)
    else:  # each adapter over all rows, the others' set to zero
        for a in range(case["G"]):
            T = (X @ A[a].float()) * ((idx == a).float() * scale[a])[:, None]
            Y = Y + T @ B[a].float()
    return Y.to(DTYPES[case["dtype"]])


def _plain_route(logits, top_k, renormalize):
    x = logits.float()
    order = torch.sort(x, dim=1, descending=True, stable=True)[1]
    ids = order[:, :top_k]
    e = torch.exp(x - x.amax(1, keepdim=True))
    w = e.gather(1, ids)
    w = w / (w if renormalize else e).sum(1, keepdim=True)
    return ids.to(torch.int32), w


def _act(x, activation):
    if activation == "silu":
        return x / (1.0 + torch.exp(-x))
    return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))


def _plain_moe(st):
    case = st["case"]
    trans, act, M, S, E = case["trans"], case["activation"], case["M"], case["top_k"], case["E"]
    ids, w = _plain_route(st["logits"], S, case["renormalize"])
    X = st["X"].float()
    Wg, Wu, Wd = st["W_gate"], st["W_up"], st["W_down"]
    if trans:
        Wg, Wu, Wd = Wg.transpose(1, 2), Wu.transpose(1, 2), Wd.transpose(1, 2)
    Y = torch.zeros_like(X)
    if M * S <= E:  # gather each pair's expert
        for s in range(S):
            e = ids[:, s].long()
            gate = (X[:, :, None] * Wg[e].float()).sum(1)
            up = (X[:, :, None] * Wu[e].float()).sum(1)
            h = _act(gate, act) * up * w[:, s:s + 1]
            Y = Y + (h[:, :, None] * Wd[e].float()).sum(1)
    else:  # each expert over all tokens, the others' weighted with zero
        for e in range(E):
            we = (w * (ids == e).float()).sum(1, keepdim=True)
            h = _act(X @ Wg[e].float(), act) * (X @ Wu[e].float()) * we
            Y = Y + h @ Wd[e].float()
    return Y.to(DTYPES[case["dtype"]])


def _plain_logprobs(st):
    top_k = st["case"]["top_k"]
    x = st["logits"].float()
    m = x.amax(1, keepdim=True)
    d = x - m
    e = torch.exp(d)
    s = e.sum(1, keepdim=True)
    log_s = torch.log(s)
    lse = (m + log_s)[:, 0]
    logp = d.gather(1, st["targets"][:, None]) - log_s
    entropy = log_s - (e * torch.where(e > 0, d, torch.zeros_like(d))).sum(1, keepdim=True) / s
    if not top_k:
        return logp[:, 0], entropy[:, 0], lse
    # order by value, ties by the lower index: one 64-bit key for both
    bits = x.view(torch.int32)
    key = torch.where(bits < 0, bits ^ 0x7fffffff, bits).to(torch.int64) * (1 << 32)
    key = key + ((1 << 32) - 1 - torch.arange(x.shape[1], device=x.device))
    ids = ((1 << 32) - 1) - (torch.topk(key, top_k, dim=1)[0] & ((1 << 32) - 1))
    return logp[:, 0], entropy[:, 0], lse, ids.to(torch.int32), d.gather(1, ids) - log_s


def _plain_logprobs_grad(st):
    x = st["logits"].float()
    logp = x - st["lse"][:, None]
    p = torch.exp(logp)
    t = st["targets"]
    gl = torch.where(t >= 0, st["g_logprobs"], torch.zeros_like(st["g_logprobs"]))
    d = -gl[:, None] * p
    d.scatter_add_(1, t.clamp(min=0)[:, None], gl[:, None])
    if st["g_entropy"] is not None:
        d = d - st["g_entropy"][:, None] * p * (logp + st["entropy"][:, None])
    return d.to(st["logits"].dtype)


def _plain(st):
    case = st["case"]
    if case["op"] == "lora":
        return _plain_lora(st)
    if case["op"] == "route":
        return _plain_route(st["logits"], case["top_k"], case["renormalize"])
    if case["op"] == "moe":
        return _plain_moe(st)
    if case["op"] == "logprobs":
        return _plain_logprobs(st)
    return _plain_logprobs_grad(st)


# ---------------------------------------------------------------------------- one pass

def run(st):
    if not own:
        return _plain(st)
    import onnx_matmul_family_amd as omm
    case = st["case"]
    if case["op"] == "lora":
        return omm.lora_matmul(st["X"], st["W"], st["A"], st["B"], st["idx"], st["scale"], st["bias"],
                               trans=case["trans"], workspace=st["ws"])[0]
    if case["op"] == "route":
        return omm.moe_route(st["logits"], case["top_k"], renormalize=case["renormalize"])
    if case["op"] == "moe":
        return omm.moe_layer(st["X"], st["logits"], case["top_k"], st["W_gate"], st["W_up"], st["W_down"],
                             renormalize=case["renormalize"], activation=case["activation"], trans=case["trans"],
                             workspace=st["ws"])[0]
    if case["op"] == "logprobs":
        out = omm.token_logprobs(st["logits"], st["targets"], top_k=case["top_k"], workspace=st["ws"])
        return out if case["top_k"] else out[:3]
    return omm.token_logprobs_grad(st["logits"], st["targets"], st["lse"], st["g_logprobs"], st["entropy"],
                                   st["g_entropy"])


# ---------------------------------------------------------------------------- definitions in 64 bits

def _exact_lora(st):
    case = st["case"]
    sub = "n" if not case["trans"] else "t"
    X, scale, idx = st["X"].double(), st["scale"].double(), st["idx"].tolist()
    W = st["W"].double()
    Y = torch.mm(X, W if sub == "n" else W.t().contiguous())
    if st["bias"] is not None:
        Y += st["bias"].double()
    for a in sorted(set(idx)):
        if a < 0:
            continue
        rows = torch.tensor([m for m, g in enumerate(idx) if g == a], device="cuda")
        A, B = st["A"][a].double(), st["B"][a].double()
        if sub == "t":
            A, B = A.t().contiguous(), B.t().contiguous()
        Y[rows] += scale[a] * torch.mm(torch.mm(X[rows], A), B)
    return Y


def _exact_route(logits, top_k, renormalize):
    x = logits.double()
    # the rank of each logit: how many come before it, by value and then by index
    ids = torch.empty((x.shape[0], top_k), dtype=torch.int64, device=x.device)
    E = x.shape[1]
    earlier = torch.arange(E, device=x.device)
    for r0 in range(0, x.shape[0], 1024):
        y = x[r0:r0 + 1024]
        before = (y[:, None, :] > y[:, :, None]) | ((y[:, None, :] == y[:, :, None]) &
                                                    (earlier[None, None, :] < earlier[None, :, None]))
        rank = before.sum(2)
        for s in range(top_k):
            ids[r0:r0 + 1024, s] = (rank == s).to(torch.int64).argmax(1)
    p = torch.softmax(x, 1).gather(1, ids)
    if renormalize:
        p = p / p.sum(1, keepdim=True)
    return ids.to(torch.int32), p


def _exact_moe(st):
    case = st["case"]
    X = st["X"].double()
    ids, w = _exact_route(st["logits"], case["top_k"], case["renormalize"])
    Y = torch.zeros_like(X)
    for e in range(case["E"]):
        rows, slots = torch.nonzero(ids == e, as_tuple=True)
        if rows.numel() == 0:
            continue
        Wg, Wu, Wd = (st[n][e].double() for n in ("W_gate", "W_up", "W_down"))
        if case["trans"]:
            Wg, Wu, Wd = Wg.t().contiguous(), Wu.t().contiguous(), Wd.t().contiguous()
        g, u = torch.mm(X[rows], Wg), torch.mm(X[rows], Wu)
        if case["activation"] == "silu":
            a = g * torch.sigmoid(g)
        else:
            a = g * 0.5 * torch.special.erfc(-g / math.sqrt(2.0))
        Y[rows] += w[rows, slots][:, None] * torch.mm(a * u, Wd)
    return Y


def _exact_logprobs(st):
    case = st["case"]
    k = case["top_k"]
    parts = []
    for r0 in range(0, case["M"], 128):
        x = st["logits"][r0:r0 + 128].double()
        lse = torch.logsumexp(x, 1, keepdim=True)
        lp = x - lse
        p = torch.exp(lp)
        ent = -torch.special.xlogy(p, p).sum(1)
        out = [lp.gather(1, st["targets"][r0:r0 + 128, None])[:, 0], ent, lse[:, 0]]
        if k:
            val, ids = torch.sort(x, dim=1, descending=True, stable=True)
            out += [ids[:, :k].to(torch.int32), (val[:, :k] - lse).contiguous()]
        parts.append(out)
    return tuple(torch.cat(c) for c in zip(*parts))


def _exact_logprobs_grad(st):
    case = st["case"]
    out = torch.empty((case["M"], case["V"]), dtype=torch.float64, device="cuda")
    for r0 in range(0, case["M"], 128):
        s = slice(r0, min(r0 + 128, case["M"]))
        x = st["logits"][s].double()
        p = torch.softmax(x, 1)
        t = st["targets"][s]
        hot = torch.arange(case["V"], device="cuda")[None, :] == t[:, None]
        gl = st["g_logprobs"][s].double() * (t >= 0)
        d = gl[:, None] * (hot.double() - p)
        if st["g_entropy"] is not None:
            lp = torch.log_softmax(x, 1)
            H = -torch.special.xlogy(p, p).sum(1, keepdim=True)
            d -= st["g_entropy"][s].double()[:, None] * p * (lp + H)
        out[s] = d
    return out


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "lora":
        return _exact_lora(st)
    if case["op"] == "route":
        return _exact_route(st["logits"], case["top_k"], case["renormalize"])
    if case["op"] == "moe":
        return _exact_moe(st)
    if case["op"] == "logprobs":
        return _exact_logprobs(st)
    return _exact_logprobs_grad(st)
