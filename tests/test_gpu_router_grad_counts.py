"""moe_route_grad with counts that several processes' batches add up to."""
import pytest
import torch

from tests.test_gpu_router_grad import case, check_grad

pytestmark = pytest.mark.gpu

om = pytest.importorskip("onnx_matmul_family_amd._omm")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    om.lib()


@pytest.mark.parametrize("E,each", [(8, 2 ** 29), (16, 2 ** 27), (64, 2 ** 31 - 200), (512, 5_000_000)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_counts_whose_sum_passes_31_bits(E, each, dt):
    """Every count fits int32; their sum is 2^31 and more."""
    x, ids, mask, g = case(40, E, 4, dt, 0.2, seed=E)
    counts = (each + torch.arange(E) % 100).to(torch.int32)
    n = 2 ** 30
    assert int(counts.long().sum()) >= 2 ** 31
    gl = torch.tensor([0.3 * n, 0.01 * n])
    tokens = torch.tensor([n], dtype=torch.int32)
    check_grad(x, ids, mask, g, True, dt, gl, counts.cuda(), tokens.cuda())
    # what the first loss alone gives: none of it is lost
    got = check_grad(x, ids, mask, None, True, dt, torch.tensor([0.3 * n, 0.0]), counts.cuda(), tokens.cuda())
    assert bool((got[mask.cuda()] != 0).any())
