"""moe_route_grad of renormalised weights whose selections lie far below the token's largest logit (indices that are
not the largest: groups, random second choices, a capacity that is used up)."""
import math

import pytest
import torch

from tests.decode_util import TORCH, U, assert_within, half_step

pytestmark = pytest.mark.gpu

om = pytest.importorskip("onnx_matmul_family_amd._omm")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    om.lib()


def renormalised(x, ids, g, dt):
    """(gradient, tolerance): w the softmax of the selections among themselves, in 64 bits.  The tolerance counts as
    route_grad of train_util does, with the span of logits below which fp32's exponential is 0."""
    x = x.double()
    M, E = x.shape
    d, s, span = torch.zeros_like(x), torch.zeros_like(x), torch.zeros((M, 1), dtype=torch.float64)
    for m in range(M):
        span[m] = min(float((x[m].max() - x[m][torch.isfinite(x[m])]).max()) if torch.isfinite(x[m]).any() else 0.0, 104.0)
        sel = [(int(e), float(v)) for e, v in zip(ids[m], g[m]) if 0 <= int(e) < E and float(x[m, int(e)]) > -math.inf]
        if not sel:
            continue
        top = max(float(x[m, e]) for e, _ in sel)
        w = [math.exp(float(x[m, e]) - top) for e, _ in sel]
        total = sum(w)
        mean = sum(a / total * v for a, (_, v) in zip(w, sel))
        size = sum(a / total * abs(v) for a, (_, v) in zip(w, sel))
        for a, (e, v) in zip(w, sel):
            d[m, e] += a / total * (v - mean)
            s[m, e] += a / total * (abs(v) + size)
    tol = U * s * (3 * (span + E + 8) + 2 * E + 32) + 1e-37
    return d, tol + half_step(dt, d.abs() + tol)


@pytest.mark.parametrize("E,k", [(8, 2), (16, 16), (24, 3), (64, 4), (65, 8), (160, 6), (257, 5), (512, 16)])
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_selections_far_below_the_largest(E, k, dt):
    gen = torch.Generator().manual_seed(E + k)
    M = 60
    x = torch.randn((M, E), generator=gen)
    # the k of the selections, 0 to 300 below the rest
    ids = torch.stack([torch.randperm(E, generator=gen)[:k] for _ in range(M)]).to(torch.int32)
    below = torch.linspace(0, 300, M)[:, None]
    if k < E:
        x.scatter_add_(1, ids.long(), -below.expand(M, k))
    else:
        x[:, 1:] -= below  # (all are selected: the first is the largest by far)
    x[5], x[6, 0] = -math.inf, -math.inf
    x[7].scatter_(0, ids[7].long(), -math.inf)  # nothing but excluded experts selected
    ids[8, 0], ids[9, 0] = -1, E
    if k > 1:
        ids[10, 1] = ids[10, 0]
        x[11, int(ids[11, 0])] = -math.inf
    x = x.to(TORCH[dt])
    g = torch.randn((M, k), generator=gen)
    got = om.moe_route_grad(x.cuda(), ids.cuda(), g.cuda(), renormalize=True)
    assert bool(torch.isfinite(got.float()).all())
    want, tol = renormalised(x, ids, g, dt)
    assert_within(got, want, tol, "gradient")
    # in place, and with padded tokens between the others
    mask = torch.rand((M,), generator=gen) >= 0.3
    y = x.cuda()
    om.moe_route_grad(y, ids.cuda(), g.cuda(), renormalize=True, token_mask=mask.cuda(), grad_logits=y)
    assert bool((y[~mask.cuda()] == 0).all()) and torch.equal(y[mask.cuda()], got[mask.cuda()])


def test_with_the_losses():
    """The losses' part beside it is what it is without the selections."""
    gen = torch.Generator().manual_seed(3)
    x = torch.randn((50, 96), generator=gen)
    ids = torch.stack([torch.randperm(96, generator=gen)[:4] for _ in range(50)]).to(torch.int32)
    x.scatter_add_(1, ids.long(), torch.full((50, 4), -120.0))
    g = torch.randn((50, 4), generator=gen)
    _, counts, tokens = om.moe_balance(x.cuda(), ids.cuda())
    gl = torch.tensor([20.0, 5.0], device="cuda")
    args = dict(counts=counts, tokens=tokens, grad_losses=gl)
    both = om.moe_route_grad(x.cuda(), ids.cuda(), g.cuda(), **args).double().cpu()
    losses = om.moe_route_grad(x.cuda(), ids.cuda(), **args).double().cpu()
    want, tol = renormalised(x, ids, g, "f32")
    # (the sum of the two parts is rounded once more)
    assert_within(both, want + losses, tol + U * (want + losses).abs() + 1e-37, "gradient")
