"""The gradient's exponentials to the last bits: its p is as good as fp32 holds l = x - lse."""
import pytest
import torch

pytestmark = pytest.mark.gpu

om = pytest.importorskip("onnx_matmul_family_amd._omm")

U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    om.lib()


@pytest.mark.parametrize("V", [1000, 40001])
def test_gradient_of_exact_differences(V):
    """x - lse is exact, so what is left is the exponential's own error (2 u), the products' (3 u), and
    ln 2 in fp32, off by 2^-28.4 of itself: |l| u / 16 is above it."""
    gen = torch.Generator().manual_seed(V)
    M = 6
    x = -torch.randint(0, 80 * 1024, (M, V), generator=gen).float() / 1024
    t = torch.zeros((M,), dtype=torch.int64)
    lse, gl = torch.zeros((M,)), torch.full((M,), 2.0)
    got = om.token_logprobs_grad(x.cuda(), t.cuda(), lse.cuda(), gl.cuda()).cpu().double()
    want = -2.0 * torch.exp(x.double())
    want[:, 0] += 2.0
    tol = U * (8 + x.double().abs() / 16) * (2.0 * torch.exp(x.double()))
    tol[:, 0] += U * 4
    assert bool(((got - want).abs() <= tol).all()), float(((got - want).abs() / tol).max())
