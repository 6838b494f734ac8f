"""moe_layer with experts that the router's mask excludes."""
import math

import pytest
import torch

from tests.decode_util import assert_within, moe
from tests.test_gpu_moe import layer_case

pytestmark = pytest.mark.gpu

om = pytest.importorskip("onnx_matmul_family_amd._omm")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    om.lib()


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("trans", [0, 1])
@pytest.mark.parametrize("M,K,F,E,k", [(5, 64, 72, 6, 3), (40, 128, 96, 5, 4), (5, 7, 5, 6, 3), (4, 512, 192, 70, 6)])
def test_layer_excluded_experts_leave_no_trace(M, K, F, E, k, dt, trans):
    """An expert whose logit is -inf adds nothing, whatever its weights hold, also where it is
    selected because fewer than top_k others are left."""
    X, logits, g, u, d = layer_case(M, K, F, E, k, dt, trans, 100 + M)
    logits[:, 0] = -math.inf
    logits[1, 2:] = -math.inf          # one left (expert 1)
    logits[2] = -math.inf              # none left
    logits[3, E - 1] = -math.inf
    want, tol = moe(X, logits, k, *[torch.cat([w[:1] * 0, w[1:]]) for w in (g, u, d)], True, "silu", trans, dt)
    g[0], u[0], d[0] = math.nan, math.inf, math.nan
    got, _ = om.moe_layer(X.cuda(), logits.cuda(), k, g.cuda(), u.cuda(), d.cuda(), trans=trans)
    assert_within(got, want, tol)
    assert bool((got[2] == 0).all())
