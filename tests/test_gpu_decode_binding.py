"""Arguments that the native binding of the decode-side operators refuses."""
import pytest
import torch

pytestmark = pytest.mark.gpu

om = pytest.importorskip("onnx_matmul_family_amd._omm")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    om.lib()


@pytest.mark.parametrize("k", [2 ** 32 + 2, -2 ** 32 + 2, 2 ** 63])
def test_selections_past_32_bits(k):
    """No wrap to a count that there is."""
    x = torch.randn((4, 16), device="cuda")
    w = torch.randn((16, 16, 16), device="cuda")
    ws = torch.empty((1 << 20,), dtype=torch.uint8, device="cuda")
    ids, p = torch.empty((4, 2), dtype=torch.int32, device="cuda"), torch.empty((4, 2), device="cuda")
    with pytest.raises(OverflowError):
        om.moe_route(x, k, indices=ids, weights=p)
    with pytest.raises(OverflowError):
        om.moe_layer(x, x, k, w, w, w, workspace=ws)
    with pytest.raises(OverflowError):
        om.token_logprobs(x, torch.zeros((4,), dtype=torch.int64, device="cuda"), top_k=k, workspace=ws)
    with pytest.raises(OverflowError):
        om.lora_matmul(x, w[0], w[:2], w[:2], torch.zeros((4,), dtype=torch.int32, device="cuda"), trans=k)


def test_status_of_each_refusal():
    x = torch.randn((4, 16), device="cuda")

    def code(f, *a, **kw):
        with pytest.raises(om.OmmError) as e:
            f(*a, **kw)
        return e.value.code

    t = torch.zeros((4,), dtype=torch.int64, device="cuda")
    assert code(om.moe_route, x, 17) == -3
    assert code(om.moe_route, x, -1) == -3
    assert code(om.moe_route, x, 2, indices=torch.empty((4, 2), device="cuda")) == -2
    assert code(om.moe_route, x.double(), 2) == -5
    assert code(om.moe_route, torch.randn((4, 513), device="cuda"), 2) == -5
    assert code(om.token_logprobs, x, t[:3]) == -3
    assert code(om.token_logprobs, x, t, top_k=17) == -3
    assert code(om.token_logprobs, x.repeat(1, 4), t, top_k=33) == -5
    assert code(om.token_logprobs_grad, x, t, x[:, 0].contiguous(), x[:, 0].contiguous(),
                grad_entropy=x[:, 0].contiguous()) == -1
    W, A, B = torch.randn((16, 16), device="cuda"), torch.randn((2, 16, 4), device="cuda"), \
        torch.randn((2, 4, 16), device="cuda")
    idx = t.to(torch.int32)
    small = torch.empty((256,), dtype=torch.uint8, device="cuda")[:16]
    assert code(om.lora_matmul, x, W, A, B, idx, workspace=small) == -6
    assert code(om.lora_matmul, x, W.to(torch.bfloat16), A, B, idx) == -2
    assert code(om.lora_matmul, x, W, A, B.transpose(1, 2).contiguous(), idx) == -3
    assert code(om.moe_layer, x, x, 2, *[torch.randn((16, 16, 16), device="cuda") for _ in range(3)],
                workspace=small) == -6


def test_no_selections():
    """top_k = 0: the router has nothing to write, the layer refuses."""
    x, w = torch.randn((4, 16), device="cuda"), torch.randn((16, 16, 16), device="cuda")
    ids, p = om.moe_route(x, 0)
    assert ids.shape == (4, 0) and p.shape == (4, 0)
    for k in (0, -1):
        with pytest.raises(om.OmmError) as e:
            om.moe_layer(x, x, k, w, w, w)
        assert e.value.code == -3
