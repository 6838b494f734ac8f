"""What lora_matmul and moe_layer hold between their two products: the fp32 values
themselves, to the last bit."""
import pytest
import torch

from tests.decode_util import TORCH

pytestmark = pytest.mark.gpu

om = pytest.importorskip("onnx_matmul_family_amd._omm")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    om.lib()


def zeros(*shape, dt):
    return torch.zeros(shape, dtype=TORCH[dt], device="cuda")


# Two middle values that differ in the last bit of fp32 only, subtracted: 1 + 2^-11 + 2^-23 and
# 1 + 2^-11.  Their summands are a step of the contraction apart, so every sum on the way is exact.

@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("trans", [0, 1])
@pytest.mark.parametrize("M,F", [(1, 8), (20, 72), (40, 256)])
def test_layer_middle_value_keeps_its_last_bit(M, F, dt, trans):
    K, E = 96, 2
    X = zeros(M, K, dt=dt)
    X[:, 0], X[:, 40], X[:, 72] = 1.0, 2.0 ** -11, 2.0 ** -23
    g, u, d = zeros(E, K, F, dt=dt), zeros(E, K, F, dt=dt), zeros(E, F, K, dt=dt)
    g[:, 0, :2] = 16.0                       # GELU(16) = 16
    u[:, [0, 40, 72], 0] = 1.0
    u[:, [0, 40], 1] = 1.0
    d[:, 0], d[:, 1] = 1.0, -1.0
    if trans:
        g, u, d = (t.transpose(1, 2).contiguous() for t in (g, u, d))
    logits = torch.zeros((M, E), device="cuda")
    got, _ = om.moe_layer(X, logits, 1, g, u, d, activation="gelu", trans=trans)
    assert bool((got.double() == 2.0 ** -19).all()), got.double().flatten()[:4]


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("trans", [0, 1])
@pytest.mark.parametrize("M", [3, 300, 700])
def test_lora_middle_value_keeps_its_last_bit(M, dt, trans):
    K, N, R, G = 256, 264, 8, 2
    X = zeros(M, K, dt=dt)
    X[:, 0], X[:, 100], X[:, 200] = 1.0, 2.0 ** -11, 2.0 ** -23
    W, A, B = zeros(K, N, dt=dt), zeros(G, K, R, dt=dt), zeros(G, R, N, dt=dt)
    A[:, [0, 100, 200], 0] = 1.0
    A[:, [0, 100], 1] = 1.0
    B[:, 0], B[:, 1] = 1.0, -1.0
    if trans:
        W, A, B = W.t().contiguous(), A.transpose(1, 2).contiguous(), B.transpose(1, 2).contiguous()
    got, _ = om.lora_matmul(X, W, A, B, torch.arange(M, device="cuda") % G, trans=trans)
    assert bool((got.double() == 2.0 ** -23).all()), got.double().flatten()[:4]
