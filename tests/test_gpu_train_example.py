"""examples/train_step.py runs, and its gradients are those of its loss."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "train_step.py")
    spec = importlib.util.spec_from_file_location("train_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("steps,tokens", [(1, 1), (3, 200), (2, 700)])
def test_runs(example, steps, tokens):
    model, history, served, plain = example.main(steps, tokens)
    assert len(history) == steps and served.shape == plain.shape
    for lp, losses in history:
        assert bool(torch.isfinite(lp)) and bool(torch.isfinite(losses).all())
    assert bool(torch.isfinite(model.vocab.float()).all()) and bool(torch.isfinite(model.router.float()).all())
    assert bool(torch.isfinite(served.float()).all())


def test_gradients(example):
    """Against autograd of the same loss in 64 bits (the fp32 model's own roundings: products of up to 2001
    terms and three of them in a row, 2^-24 of their terms each, far below 1e-4 of the largest gradient)."""
    model = example.Model(dtype=torch.float32)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    tokens = torch.randint(0, 2001, (90,), generator=gen, device="cuda")
    mask = torch.arange(90, device="cuda") % 5 != 4
    targets = torch.where(mask, tokens * 7 % 2001, -1)
    logits, saved = example.forward(model, tokens, mask)
    got, logprobs = example.gradients(model, logits, targets, saved, balance=0.5, z=0.05)

    d = {n: getattr(model, n).double().cpu() for n in ("embed", "W", "router", "gate", "up", "down", "vocab")}
    d["router"].requires_grad_(True)
    d["vocab"].requires_grad_(True)
    ids, keep = saved["ids"].cpu().long(), mask.cpu()
    h = d["embed"][tokens.cpu()] @ d["W"]
    route = h @ d["router"]
    p = torch.softmax(route, 1)
    w = p.gather(1, ids)
    w = w / w.sum(1, keepdim=True)
    y = h.clone()
    for s in range(ids.shape[1]):
        e = ids[:, s]
        a = torch.nn.functional.silu((h[:, None] @ d["gate"][e])[:, 0]) * (h[:, None] @ d["up"][e])[:, 0]
        y = y + w[:, s:s + 1] * (a[:, None] @ d["down"][e])[:, 0]
    lp = torch.log_softmax(y @ d["vocab"], 1)
    n = int(keep.sum())
    loss = -lp[keep].gather(1, targets.cpu()[keep][:, None]).sum() / n
    f = torch.bincount(ids[keep].reshape(-1), minlength=16).double() / (n * ids.shape[1])
    loss = loss + 0.5 * 16 * (f * p[keep].mean(0)).sum() + 0.05 * (torch.logsumexp(route[keep], 1) ** 2).mean()
    want = torch.autograd.grad(loss, [d["vocab"], d["router"]])
    for g, x in zip((got["vocab"], got["router"]), want):
        assert float((g.double().cpu() - x).abs().max()) <= 1e-4 * float(x.abs().max())
