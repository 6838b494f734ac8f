"""The decode-side operators on another stream than the caller's: the memory that a call
allocates is nobody else's while its kernels run, dropped workspaces and outputs among it."""
import pytest
import torch

from tests.test_gpu_lora import case as lora_case
from tests.test_gpu_moe import layer_case

pytestmark = pytest.mark.gpu

om = pytest.importorskip("onnx_matmul_family_amd._omm")

WAIT = 40_000_000  # clock ticks that keep a stream busy while the host goes on (20 ms or so)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    om.lib()


def rows(M, V):
    gen = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn((M, V), generator=gen, device="cuda").to(torch.bfloat16)
    return x, torch.randint(0, V, (M,), generator=gen, device="cuda")


def lora_call(M):
    c = [t.cuda() for t in lora_case(M, 1024, 1032, 16, 4, "bf16", 0, 1)]
    return lambda s: om.lora_matmul(*c, stream=s)[:1], om.lora_matmul_workspace_size(M, 1024, 1032, 16, torch.bfloat16)


def layer_call(M):
    X, logits, g, u, d = [t.cuda() for t in layer_case(M, 512, 256, 8, 2, "bf16", 0, 2)]
    return (lambda s: om.moe_layer(X, logits, 2, g, u, d, stream=s)[:1],
            om.moe_layer_workspace_size(M, 512, 256, 8, 2))


def logprobs_call(M):
    x, t = rows(M, 131072)
    return lambda s: om.token_logprobs(x, t, top_k=5, stream=s), om.token_logprobs_workspace_size(M, 131072, 5)


def grad_call(M):
    x, t = rows(M, 9001)
    _, H, lse, _, _ = om.token_logprobs(x, t)
    return lambda s: (om.token_logprobs_grad(x, t, lse, H, H, lse, stream=s),), x.numel() * 2


def route_call(M):
    x, _ = rows(M, 64)
    return lambda s: om.moe_route(x, 8, stream=s), M * 32


CALLS = [(lora_call, 5), (lora_call, 43), (lora_call, 700), (layer_call, 3), (layer_call, 40), (logprobs_call, 1),
         (logprobs_call, 40), (grad_call, 30), (route_call, 1000)]


@pytest.mark.parametrize("make,M", CALLS)
def test_tensors_made_after_the_call(make, M):
    """The stream is busy, so the call's kernels run after these tensors were made and filled."""
    call, size = make(M)
    want = [t.clone() for t in call(None)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(WAIT)
    got = call(s)                                     # (the workspace, if any, is dropped here)
    mine = [torch.full((max(size, 256),), 77, dtype=torch.uint8, device="cuda") for _ in range(6)]
    mine += [torch.full_like(t, 3) for t in want]
    torch.cuda.current_stream().synchronize()
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for t in mine[:6]:
        assert bool((t == 77).all())
    for t in mine[6:]:
        assert bool((t == 3).all())


@pytest.mark.parametrize("make,M", CALLS)
def test_tensors_freed_before_the_call(make, M):
    """The caller's stream is busy, so what it still has to read of freed tensors must not be written."""
    call, size = make(M)
    want = [t.clone() for t in call(None)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(WAIT)
    old = [torch.full((max(size, 256),), 77, dtype=torch.uint8, device="cuda")] + [torch.full_like(t, 3) for t in want]
    kept = [t.clone() for t in old]
    del old
    got = call(s)
    s.synchronize()
    torch.cuda.current_stream().synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    assert bool((kept[0] == 77).all())
    for t in kept[1:]:
        assert bool((t == 3).all())


def test_outputs_freed_while_the_caller_still_reads_them():
    call, _ = logprobs_call(40)
    want = [t.clone() for t in call(None)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        got = call(s)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda._sleep(WAIT // 4)
        copies = [t.clone() for t in got]
        del got
        with torch.cuda.stream(s):                    # takes what is free on s
            for t in want:
                torch.full_like(t, 3)
        torch.cuda.synchronize()
        for a, b in zip(copies, want):
            assert torch.equal(a, b)
