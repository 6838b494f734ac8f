"""The decode-side operators stay within the workspace size that they state, and read
nothing of what it held."""
import pytest
import torch

from tests.decode_util import TORCH
from tests.test_gpu_lora import case as lora_case
from tests.test_gpu_moe import layer_case

pytestmark = pytest.mark.gpu

om = pytest.importorskip("onnx_matmul_family_amd._omm")

GUARD = 1 << 16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    om.lib()


def within(size, call):
    """call(workspace) twice, over workspaces of other contents: the same bits, nothing written past the end."""
    outs = []
    for fill in (0, 255):
        buf = torch.full((size + GUARD,), fill, dtype=torch.uint8, device="cuda")
        buf[size:] = 90
        outs.append([t.clone() for t in call(buf[:size])])
        assert bool((buf[size:] == 90).all())
    for a, b in zip(*outs):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("trans", [0, 1])
@pytest.mark.parametrize("M,K,N,R,G", [
    (1, 512, 264, 16, 4), (16, 4096, 520, 3, 4), (43, 1032, 4104, 24, 5), (64, 64, 64, 256, 2), (257, 264, 520, 16, 5),
    (700, 128, 264, 4, 3), (700, 128, 264, 129, 3), (513, 520, 392, 200, 3), (1024, 64, 16384, 40, 3),
    (700, 129, 267, 13, 3), (50, 7, 30, 5, 2), (65536, 72, 40, 16, 5), (65601, 64, 72, 4, 5), (65601, 33, 41, 9, 3)])
def test_lora(M, K, N, R, G, dt, trans):
    c = [t.cuda() for t in lora_case(M, K, N, R, G, dt, trans, 3)]
    within(om.lora_matmul_workspace_size(M, K, N, R, TORCH[dt]),
           lambda ws: om.lora_matmul(*c, trans=trans, workspace=ws)[:1])


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("trans", [0, 1])
@pytest.mark.parametrize("M,K,F,E,k", [(1, 512, 256, 8, 3), (40, 264, 1000, 16, 4), (64, 128, 96, 4, 4), (3, 2778, 192, 2, 1),
                                       (5, 7, 60, 6, 3), (2, 64, 0, 4, 2)])
def test_layer(M, K, F, E, k, dt, trans):
    X, logits, g, u, d = [t.cuda() for t in layer_case(M, K, max(F, 1), E, k, dt, trans, 4)]
    if F == 0:
        g, u, d = (t[:, :0].contiguous() if (n == 2) != bool(trans) else t[:, :, :0].contiguous()
                   for n, t in enumerate((g, u, d)))
    within(om.moe_layer_workspace_size(M, K, F, E, k),
           lambda ws: om.moe_layer(X, logits, k, g, u, d, trans=trans, workspace=ws)[:1])


@pytest.mark.parametrize("M,V,k", [(1, 131072, 5), (3, 50001, 32), (511, 16385, 0), (40, 20000, 7)])
def test_logprobs(M, V, k):
    x = torch.randn((M, V), device="cuda").to(torch.bfloat16)
    t = torch.randint(0, V, (M,), device="cuda")
    size = om.token_logprobs_workspace_size(M, V, k)
    assert size > 0
    within(size, lambda ws: om.token_logprobs(x, t, top_k=k, workspace=ws))
