"""moe_layer without hidden columns."""
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


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("trans", [0, 1])
@pytest.mark.parametrize("M,K,E,k", [(1, 64, 4, 2), (5, 7, 3, 3), (40, 136, 2, 1)])
def test_layer_without_hidden_columns(M, K, E, k, dt, trans):
    """F = 0: an empty sum."""
    t = TORCH[dt]
    up, down = ((E, 0, K), (E, K, 0)) if trans else ((E, K, 0), (E, 0, K))
    Y = torch.full((M, K), 9.0, dtype=t, device="cuda")
    om.moe_layer(torch.randn((M, K), device="cuda").to(t), torch.randn((M, E), device="cuda"), k,
                 torch.empty(up, dtype=t, device="cuda"), torch.empty(up, dtype=t, device="cuda"),
                 torch.empty(down, dtype=t, device="cuda"), trans=trans, Y=Y)
    assert bool((Y == 0).all())
