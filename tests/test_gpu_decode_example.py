"""examples/decode_step.py runs, and what its calls hand to each other fits."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def example():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decode_step.py")
    spec = importlib.util.spec_from_file_location("decode_step", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("requests,tokens", [(1, 3), (6, 8), (20, 16)])
def test_decode_step(example, requests, tokens):
    new, lps, before, after = example.main(requests, tokens)
    assert new.shape == (tokens, requests) and bool((new >= 0).all())
    # the same tokens scored in one batch (over 64 rows through the grouped products): bf16 roundings of
    # logits up to 16 (a step of 2^-4) and of the layer's output move a log probability by less than 0.5
    assert bool(((lps.t().reshape(-1) - before).abs() < 0.5).all())
    assert float(after.mean()) > float(before.mean())
