"""The decode-side operators together, as a serving process and a policy update use them.

A one-block model with random weights: a projection with a low-rank adapter per
request, a mixture of experts, a vocabulary projection.  `generate` decodes a
batch of requests token by token; `score` runs whole sequences at once, with the
expert products of a long batch, and `update` takes one policy-gradient step on
the vocabulary projection from the tokens' log probabilities and entropy.

    python examples/decode_step.py [--tokens 8] [--requests 6]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import onnx_matmul_family_amd as omm  # noqa: E402


class Model:
    def __init__(self, width=512, experts=16, top_k=4, hidden=256, vocab=8001, adapters=5, rank=16, seed=0,
                 dtype=torch.bfloat16):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)

        def normal(*shape, std):
            return torch.randn(shape, generator=gen, device="cuda").mul_(std).to(dtype)

        self.top_k = top_k
        self.embed = normal(vocab, width, std=1.0)
        self.W = normal(width, width, std=width ** -0.5)
        self.A = normal(adapters, width, rank, std=width ** -0.5)
        self.B = normal(adapters, rank, width, std=rank ** -0.5)
        self.scale = torch.rand((adapters,), generator=gen, device="cuda") + 0.5
        self.router = normal(width, experts, std=2 * width ** -0.5)
        self.gate = normal(experts, width, hidden, std=width ** -0.5)
        self.up = normal(experts, width, hidden, std=width ** -0.5)
        self.down = normal(experts, hidden, width, std=hidden ** -0.5)
        self.vocab = normal(width, vocab, std=3 * width ** -0.5)

    def experts(self, h):
        """The expert layer: one call for a few tokens, the grouped products for a long batch."""
        logits = omm.matmul(h, self.router)
        if h.shape[0] <= 64:
            return omm.moe_layer(h, logits, self.top_k, self.gate, self.up, self.down)[0]
        ids, w = omm.moe_route(logits, self.top_k)
        gate, up = (omm.grouped_matmul(h, x, ids)[0].float() for x in (self.gate, self.up))
        inner = (torch.nn.functional.silu(gate) * up * w[:, :, None]).to(h.dtype)
        M, S, F = inner.shape
        out = omm.grouped_matmul(inner.view(M * S, F), self.down, ids.view(M * S, 1))[0]
        return out.view(M, S, -1).float().sum(1).to(h.dtype)

    def hidden(self, tokens, adapters):
        x = self.embed[tokens]
        h, _ = omm.lora_matmul(x, self.W, self.A, self.B, adapters, self.scale)
        return h + self.experts(h)

    def logits(self, h):
        return omm.matmul(h, self.vocab)


def generate(model, tokens, adapters, steps, alternatives=5):
    """Greedy decoding.  tokens (M): the last token of each request; adapters (M): its adapter or -1.
    Returns the new tokens (steps, M) and their log probabilities."""
    out, lps = [], []
    for _ in range(steps):
        logits = model.logits(model.hidden(tokens, adapters))
        _, _, _, ids, lp = omm.token_logprobs(logits, tokens, top_k=alternatives)
        tokens = ids[:, 0].contiguous()  # the most likely one; the others are what a client is shown
        out.append(tokens)
        lps.append(lp[:, 0])
    return torch.stack(out), torch.stack(lps)


def score(model, context, targets, adapters):
    """Log probabilities of targets (T), the hidden states and what the gradient needs."""
    h = model.hidden(context, adapters)
    logits = model.logits(h)
    lp, entropy, lse, _, _ = omm.token_logprobs(logits, targets)
    return lp, (h, logits, targets, lse, entropy)


def update(model, saved, advantage, entropy_weight=0.01, rate=0.5):
    """One step up sum(advantage * logprob + entropy_weight * entropy), on the vocabulary projection."""
    h, logits, targets, lse, entropy = saved
    n = h.shape[0]
    g = omm.token_logprobs_grad(logits, targets, lse, advantage / n, entropy,
                                torch.full_like(advantage, entropy_weight / n))
    omm.gemm(h, g, model.vocab, alpha=rate, beta=1.0, transA=1, Y=model.vocab)
    return g


def main(requests=6, tokens=8):
    model = Model()
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1)
    adapters = torch.randint(-1, 5, (requests,), generator=gen, device="cuda", dtype=torch.int32)
    start = torch.randint(0, 8001, (requests,), generator=gen, device="cuda", dtype=torch.int32)
    new, lps = generate(model, start, adapters, tokens)

    # the generated sequences scored in one call, their likelihood raised by one step
    context = torch.cat([start[None], new[:-1]]).t().reshape(-1)
    targets = new.t().reshape(-1).contiguous()
    rows = adapters.repeat_interleave(tokens)
    before, saved = score(model, context, targets, rows)
    update(model, saved, torch.ones_like(before))
    after, _ = score(model, context, targets, rows)
    return new, lps, before, after


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    ap.add_argument("--requests", type=int, default=6)
    ap.add_argument("--tokens", type=int, default=8)
    a = ap.parse_args()
    new, lps, before, after = main(a.requests, a.tokens)
    print("tokens of request 0:", new[:, 0].tolist())
    print("their log probabilities:", ["%.3f" % v for v in lps[:, 0].tolist()])
    print("mean log probability of all: %.4f, after one step %.4f" % (float(before.mean()), float(after.mean())))
