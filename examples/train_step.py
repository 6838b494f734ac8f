"""The operators that train, balance and quantise, as a training loop and the server after it use them.

A one-block model with random weights: a projection, a mixture of experts, a vocabulary
projection.  `step` runs a padded batch forward with the router's losses, takes the
gradients of the vocabulary projection and of the router by the package's gradient calls
and products, and steps along their orthogonalised momenta.  `Served` is the trained
model with its two projections in 8 bits.

    python examples/train_step.py [--steps 3] [--tokens 200]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import onnx_matmul_family_amd as omm  # noqa: E402


class Model:
    def __init__(self, width=256, experts=16, top_k=4, hidden=128, vocab=2001, seed=0, dtype=torch.bfloat16):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)

        def normal(*shape, std):
            return torch.randn(shape, generator=gen, device="cuda").mul_(std).to(dtype)

        self.top_k = top_k
        self.embed = normal(vocab, width, std=1.0)
        self.W = normal(width, width, std=width ** -0.5)
        self.router = normal(width, experts, std=2 * width ** -0.5)
        self.gate = normal(experts, width, hidden, std=width ** -0.5)
        self.up = normal(experts, width, hidden, std=width ** -0.5)
        self.down = normal(experts, hidden, width, std=hidden ** -0.5)
        self.vocab = normal(width, vocab, std=width ** -0.5)
        self.momenta = {"vocab": None, "router": None}


def forward(model, tokens, mask=None):
    """Logits (T, vocab) and what the gradients need."""
    h = omm.matmul(model.embed[tokens], model.W)
    route = omm.matmul(h, model.router)
    ids, w = omm.moe_route(route, model.top_k)
    losses, counts, counted = omm.moe_balance(route, ids, token_mask=mask)
    gate, up = (omm.grouped_matmul(h, x, ids)[0].float() for x in (model.gate, model.up))
    inner = (torch.nn.functional.silu(gate) * up).to(h.dtype)
    T, S, F = inner.shape
    outs = omm.grouped_matmul(inner.view(T * S, F), model.down, ids.view(T * S, 1))[0].view(T, S, -1)
    y = (h.float() + (w[:, :, None] * outs.float()).sum(1)).to(h.dtype)
    return omm.matmul(y, model.vocab), dict(h=h, route=route, ids=ids, outs=outs, y=y, losses=losses, counts=counts,
                                            counted=counted, mask=mask)


def gradients(model, logits, targets, saved, balance=0.01, z=0.001):
    """Of the mean negative log probability of the targets (outside [0, vocab): not counted) plus balance and z
    times the router's losses, with respect to the vocabulary projection and the router."""
    logprobs, _, lse, _, _ = omm.token_logprobs(logits, targets)
    g = torch.full_like(logprobs, -1.0) / saved["counted"]
    dlogits = omm.token_logprobs_grad(logits, targets, lse, g)
    dy = omm.gemm(dlogits, model.vocab, transB=1)
    dw = (saved["outs"].float() * dy.float()[:, None, :]).sum(2)
    droute = omm.moe_route_grad(saved["route"], saved["ids"], dw, token_mask=saved["mask"], counts=saved["counts"],
                                tokens=saved["counted"], grad_losses=torch.tensor([balance, z], device=dw.device))
    return {"vocab": omm.gemm(saved["y"], dlogits, transA=1), "router": omm.gemm(saved["h"], droute, transA=1)}, logprobs


def step(model, tokens, targets, mask=None, rate=0.02, momentum=0.9):
    """One step down; returns the mean log probability of the counted targets and the router's losses before it."""
    logits, saved = forward(model, tokens, mask)
    grads, logprobs = gradients(model, logits, targets, saved)
    for name, g in grads.items():
        m = model.momenta[name]
        m = g if m is None else torch.add(g, m, alpha=momentum)
        model.momenta[name] = m
        weight = getattr(model, name)
        update, _ = omm.orthogonalize(m)
        weight.sub_(update, alpha=rate)
    return logprobs.sum() / saved["counted"], saved["losses"]


class Served:
    """The model with its projections in int8, a scale for each output channel and each token."""

    def __init__(self, model):
        self.model = model
        self.W, self.W_scale = omm.quantize_rows(model.W.t().contiguous())
        self.vocab, self.vocab_scale = omm.quantize_rows(model.vocab.t().contiguous())

    def logits(self, tokens):
        m = self.model
        h, _ = omm.int8_matmul(m.embed[tokens], self.W, self.W_scale)
        y, _ = omm.moe_layer(h, omm.matmul(h, m.router), m.top_k, m.gate, m.up, m.down)
        return omm.int8_matmul(h + y, self.vocab, self.vocab_scale)[0]


def main(steps=3, tokens=200, dtype=torch.bfloat16):
    model = Model(dtype=dtype)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    history = []
    for _ in range(steps):
        context = torch.randint(0, 2001, (tokens,), generator=gen, device="cuda")
        mask = torch.arange(tokens, device="cuda") % 8 != 7  # (padding)
        targets = torch.where(mask, context * 7 % 2001, -1)
        history.append(step(model, context, targets, mask))
    served = Served(model)
    few = torch.randint(0, 2001, (5,), generator=gen, device="cuda")
    return model, history, served.logits(few), forward(model, few)[0]


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=3)
    ap.add_argument("--tokens", type=int, default=200)
    a = ap.parse_args()
    _, history, served, plain = main(a.steps, a.tokens)
    for lp, losses in history:
        print("mean log probability %.4f, balance loss %.4f, z loss %.4f" % (float(lp), *losses.tolist()))
    print("logits in 8 bits off by %.4f of %.4f" % (float((served - plain).float().abs().max()), float(plain.float().abs().max())))
