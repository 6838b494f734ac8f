"""Infinities, NaN and zeros between the two products of lora_matmul and moe_layer."""
import math

import pytest
import torch

from tests.decode_util import assert_within, lora, moe
from tests.test_gpu_lora import case as lora_case, run as run_lora
from tests.test_gpu_moe import layer_case

pytestmark = pytest.mark.gpu

om = pytest.importorskip("onnx_matmul_family_amd._omm")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    om.lib()


def check_infinite(got, want, tol, inf):
    got = got.double().cpu()
    assert torch.equal(got[inf], want[inf]), (got[inf][:4], want[inf][:4])
    assert_within(got[~inf], want[~inf], tol[~inf])


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("trans", [0, 1])
@pytest.mark.parametrize("M,K,F,E,k", [(2, 64, 72, 3, 1), (20, 256, 200, 4, 2), (40, 128, 96, 4, 3), (3, 7, 5, 2, 1)])
def test_layer_infinite_down_weights(M, K, F, E, k, dt, trans):
    """An infinity times a middle value is an infinity of the product's sign, not NaN."""
    X, logits, g, u, d = layer_case(M, K, F, E, k, dt, trans, 80 + M)
    cols = torch.arange(0, K, 3)
    for e in range(E):
        for i, c in enumerate(cols.tolist()):
            v = -math.inf if i % 2 else math.inf
            d[(e, c, (i + e) % F) if trans else (e, (i + e) % F, c)] = v
    want, tol = moe(X, logits, k, g, u, d, True, "silu", trans, dt)
    # (a sum of infinities of both signs is NaN in either)
    got, _ = om.moe_layer(X.cuda(), logits.cuda(), k, g.cuda(), u.cuda(), d.cuda(), trans=trans)
    inf = torch.zeros((M, K), dtype=torch.bool)
    inf[:, cols] = True
    keep = ~want.isnan()
    assert torch.equal(got.cpu().isnan(), want.isnan())
    check_infinite(got.cpu()[keep], want[keep], tol[keep], inf[keep])
    assert int(want.isinf().sum()) > 0


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("trans", [0, 1])
@pytest.mark.parametrize("M", [30, 300, 700, 1100])
def test_lora_infinite_adapter_weights(M, dt, trans):
    c = lora_case(M, 128, 264, 16, 4, dt, trans, 90)
    cols = torch.arange(0, 264, 5)
    for g in range(4):
        for i, n in enumerate(cols.tolist()):
            c[3][(g, n, (i + g) % 16) if trans else (g, (i + g) % 16, n)] = -math.inf if i % 2 else math.inf
    want, tol = lora(*c, trans, dt)
    got, _ = run_lora(c, trans)
    inf = torch.zeros((M, 264), dtype=torch.bool)
    inf[:, cols] = True
    inf &= (c[4] >= 0)[:, None]
    assert bool(want[inf].isinf().all())
    check_infinite(got, want, tol, inf)


def test_zero_middle_values_stay_zero():
    """Nothing is added for a middle value of 0: scale 0, and an activation of 0."""
    for M in (5, 700):
        X, W, A, B, idx, s, _ = lora_case(M, 128, 264, 16, 4, "bf16", 1, 91)
        got, _ = run_lora((X, W * 0, A, B, idx, s * 0, None), 1)
        assert bool((got == 0).all())
    X, logits, g, u, d = layer_case(5, 64, 72, 4, 2, "bf16", 0, 92)
    got, _ = om.moe_layer(X.cuda(), logits.cuda(), 2, g.cuda() * 0, u.cuda(), d.cuda())
    assert bool((got == 0).all())


@pytest.mark.parametrize("trans", [0, 1])
def test_middle_values_of_nan_stay_nan(trans):
    for dt in ("bf16", "f16", "f32"):
        for M in (30, 700):
            c = lora_case(M, 128, 264, 16, 2, dt, trans, 93)
            c[4][:] = torch.arange(M) % 2
            c[2][1] = math.nan
            got, _ = run_lora(c, trans)
            want, tol = lora(*c, trans, dt)
            assert_within(got, want, tol)
            assert bool(got[1::2].isnan().all())


def test_middle_values_past_fp16_beside_an_infinity():
    """fp16 rows of an infinity and of finite values beyond 65504 of the other sign: the infinity stays."""
    for M in (30, 700):
        K, N, R = 128, 264, 16
        X = torch.zeros((M, K), dtype=torch.float16)
        X[:, 0] = 1.0
        X[::2, 1] = 1.0
        A = torch.zeros((1, K, R), dtype=torch.float16)
        A[0, 0] = -60000.0
        s = torch.tensor([1e4])            # T = -6e8, and +inf in column 0 of the even rows
        A[0, 0, 0], A[0, 1, 0] = 0.0, math.inf
        A[0, 1, 1:] = 0.0
        B = torch.full((1, R, N), 2.0 ** -20, dtype=torch.float16)
        W = torch.zeros((K, N), dtype=torch.float16)
        got, _ = run_lora((X, W, A, B, torch.zeros((M,), dtype=torch.int64), s, None), 0)
        # the odd rows have 0 * inf = NaN in column 0
        assert bool((got[::2] == math.inf).all()) and bool(got[1::2].isnan().all())
