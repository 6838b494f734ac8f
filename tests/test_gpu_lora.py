"""lora_matmul on the GPU against the 64-bit form of tests/decode_util.py
(which derives the bounds)."""
import pytest
import torch

from tests.decode_util import TORCH, assert_within, draw, lora

pytestmark = pytest.mark.gpu

om = pytest.importorskip("onnx_matmul_family_amd._omm")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    om.lib()


def case(M, K, N, R, G, dt, trans, seed, bias=True, scale=True, runs=False):
    gen = torch.Generator().manual_seed(seed)
    X = draw(gen, (M, K), 1.0, dt)
    W = draw(gen, (N, K) if trans else (K, N), max(K, 1) ** -0.5, dt)
    A = draw(gen, (G, R, K) if trans else (G, K, R), max(K, 1) ** -0.5, dt)
    B = draw(gen, (G, N, R) if trans else (G, R, N), max(R, 1) ** -0.5, dt)
    idx = torch.randint(-1, G, (M,), generator=gen) if G else torch.full((M,), -1)
    if runs:
        idx = torch.sort(idx)[0]
    s = torch.rand((G,), generator=gen) * 2 - 0.5 if scale else None
    return X, W, A, B, idx, s, draw(gen, (N,), 0.5, dt) if bias else None


def run(c, trans, **kw):
    d = [t.cuda() if t is not None else None for t in c]
    return om.lora_matmul(*d, trans=trans, **kw)


def check(c, trans, dt, **kw):
    want, tol = lora(*c, trans, dt)
    got, _ = run(c, trans, **kw)
    torch.cuda.synchronize()
    assert_within(got, want, tol)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("trans", [0, 1])
@pytest.mark.parametrize("M,K,N,R,G", [
    (1, 512, 256, 16, 4), (1, 4096, 1024, 8, 2), (2, 64, 64, 4, 1), (7, 200, 136, 24, 3), (16, 256, 512, 64, 16),
    (17, 264, 128, 16, 5), (33, 1032, 72, 32, 8), (64, 320, 320, 16, 64), (5, 100, 50, 3, 3), (3, 7, 5, 1, 2),
    (1, 1, 1, 1, 1), (65, 256, 256, 16, 4), (130, 264, 392, 40, 7), (200, 100, 70, 5, 3), (300, 512, 512, 64, 2),
    (9, 2048, 4104, 17, 4), (64, 64, 64, 256, 2), (100, 64, 64, 256, 2)])
def test_lora(M, K, N, R, G, dt, trans):
    check(case(M, K, N, R, G, dt, trans, M + K + N + R, bias=bool(N % 3), scale=bool(M % 2), runs=M > 64 and R > 16),
          trans, dt)


@pytest.mark.parametrize("M", [4, 100])
@pytest.mark.parametrize("trans", [0, 1])
def test_lora_no_adapter_out_of_range_and_empty(M, trans):
    """Indices outside [0, G) on either side select none; no adapters at all; rank 0; K = 0."""
    c = list(case(M, 128, 96, 8, 3, "bf16", trans, 1))
    c[4] = torch.tensor([-1, 3, -2 ** 31, 2 ** 31 - 1])[torch.arange(M) % 4]
    check(c, trans, "bf16")
    c[4] = torch.tensor([2 ** 32, -2 ** 40, 1, 2 ** 62])[torch.arange(M) % 4]  # int64, no wrap to a valid index
    check(c, trans, "bf16")
    check(case(M, 128, 96, 8, 0, "bf16", trans, 2), trans, "bf16")
    check(case(M, 128, 96, 0, 3, "bf16", trans, 3), trans, "bf16")
    check(case(M, 0, 96, 8, 3, "bf16", trans, 4), trans, "bf16")


@pytest.mark.parametrize("M", [6, 80])
@pytest.mark.parametrize("trans", [0, 1])
def test_lora_int32_indices_unaligned_canaries_stream(M, trans):
    c = list(case(M, 128, 136, 16, 4, "bf16", trans, 12))
    want, tol = lora(*c, trans, "bf16")
    d = [t.cuda() for t in c]
    d[4] = d[4].to(torch.int32)
    for i in (1, 2, 3):  # weights one element past an aligned base
        b = torch.zeros(d[i].numel() + 1, dtype=torch.bfloat16, device="cuda")
        b[1:].view(d[i].shape).copy_(d[i])
        d[i] = b[1:].view(d[i].shape)
    out = torch.full((M + 2, 136), 9.0, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    om.lora_matmul(*d, trans=trans, Y=out[1:-1], stream=s)
    s.synchronize()
    assert_within(out[1:-1], want, tol)
    assert bool((out[0] == 9).all()) and bool((out[-1] == 9).all())


@pytest.mark.parametrize("M", [1, 20, 150])
def test_lora_repeats_bit_for_bit(M):
    d = [t.cuda() for t in case(M, 512, 512, 16, 6, "bf16", 1, M)]
    Y, ws = om.lora_matmul(*d, trans=1)
    first = Y.clone()
    ws.fill_(255)
    for _ in range(5):
        Y2, _ = om.lora_matmul(*d, trans=1, workspace=ws)
        assert torch.equal(Y2.view(torch.int16), first.view(torch.int16))


@pytest.mark.parametrize("trans", [0, 1])
def test_lora_rows_do_not_mix(trans):
    """NaN in one row, or in the adapter of other rows only, stays there."""
    for M in (12, 90):
        c = case(M, 128, 128, 16, 4, "bf16", trans, 30)
        c[4][:] = torch.arange(M) % 3  # adapter 3 is in nobody's use
        c[2][3] = float("nan")
        c[3][3] = float("nan")
        want, tol = lora(*c, trans, "bf16")
        c[0][5] = float("nan")
        got, _ = run(c, trans)
        keep = torch.arange(M) != 5
        assert_within(got[keep.cuda()], want[keep], tol[keep])
        assert bool(got[5].isnan().all())


def test_lora_past_32_bit_offsets():
    M, K, N = 70000, 64, 32768  # 2.3e9 outputs
    c = case(M, K, N, 8, 4, "bf16", 1, 40)
    got, _ = run(c, 1)
    sel = torch.tensor([0, 1, M // 2, M - 2, M - 1])
    want, tol = lora(c[0][sel], c[1], c[2], c[3], c[4][sel], c[5], c[6], 1, "bf16")
    assert_within(got[sel.cuda()], want, tol)
