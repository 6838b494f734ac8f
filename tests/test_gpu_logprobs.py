"""token_logprobs and its gradient on the GPU against the 64-bit forms of
tests/decode_util.py (which derives the bounds)."""
import math

import pytest
import torch

from tests.decode_util import TORCH, assert_within, logprobs, logprobs_grad

pytestmark = pytest.mark.gpu

om = pytest.importorskip("onnx_matmul_family_amd._omm")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    om.lib()


def rows(M, V, dt, seed, masked=0.0, std=3.0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((M, V), generator=gen) * std
    x.scatter_add_(1, torch.randint(0, V, (M, 2), generator=gen), torch.full((M, 2), 9.0))
    if masked:
        x.masked_fill_(torch.rand((M, V), generator=gen) < masked, -math.inf)
    t = torch.randint(-1, V, (M,), generator=gen)
    return x.to(TORCH[dt]), t


def check(x, t, k, what=""):
    want, tol = logprobs(x, t, k)
    got = om.token_logprobs(x.cuda(), t.cuda(), top_k=k)
    torch.cuda.synchronize()
    assert torch.equal(got[3].cpu().to(torch.int64), want[3]), what
    for i in (0, 1, 2, 4):
        assert_within(got[i], want[i], tol[i], "%s output %d" % (what, i))
    return got


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,V,k", [(1, 1, 1), (3, 2, 2), (2, 7, 0), (5, 64, 32), (4, 255, 5), (1, 4096, 20),
                                   (1, 131072, 5), (3, 50001, 20), (7, 8193, 32), (520, 1001, 1), (600, 5003, 20)])
def test_logprobs(M, V, k, dt):
    x, t = rows(M, V, dt, M * 1000 + V + k)
    check(x, t, k)


@pytest.mark.parametrize("masked", [0.5, 0.999])
@pytest.mark.parametrize("M,V", [(2, 300), (3, 40007), (513, 2050)])
def test_logprobs_masked(M, V, masked):
    x, t = rows(M, V, "bf16", V, masked)
    check(x, t, min(20, V))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [9, 4100, 70001])
def test_logprobs_ties_and_special_rows(V, dt):
    """Equal logits, ascending and descending rows, rows of -inf, the type's lowest value, NaN and +inf."""
    x = torch.zeros((10, V))
    x[1] = torch.arange(V) / 64.0
    x[2] = -torch.arange(V) / 64.0
    x[3] = -math.inf
    x[4, V // 2:] = -math.inf
    x[5] = torch.finfo(TORCH[dt]).min
    x[5, V - 1] = 0.0
    x[6] = -math.inf
    x[6, V - 2] = 1.5
    x[7, V // 3] = math.nan
    x[8, [0, V - 1]] = math.inf
    x[9] = torch.arange(V) % 2 * -0.0  # zeros of both signs tie
    t = torch.tensor([0, V - 1, 0, 1, V - 1, 0, V - 2, 0, 0, V])
    check(x.to(TORCH[dt]), t, min(9, V), dt)


@pytest.mark.parametrize("off", [1, 3])
def test_logprobs_unaligned_base_int32_targets_and_stream(off):
    x, t = rows(5, 9001, "bf16", 5)
    buf = torch.zeros(x.numel() + off, dtype=torch.bfloat16, device="cuda")
    v = buf[off:].view(5, 9001)
    v.copy_(x)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = om.token_logprobs(v, t.to(torch.int32).cuda(), top_k=7, stream=s)
    s.synchronize()
    want, tol = logprobs(x, t, 7)
    assert torch.equal(got[3].cpu().to(torch.int64), want[3])
    for i in (0, 1, 2, 4):
        assert_within(got[i], want[i], tol[i], str(i))


def grad_case(M, V, dt, seed, masked=0.0):
    x, t = rows(M, V, dt, seed, masked)
    want, _ = logprobs(x, t, 0)
    gen = torch.Generator().manual_seed(seed + 1)
    return x, t, want[2].float(), want[1].float(), torch.randn((M,), generator=gen), torch.randn((M,), generator=gen)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,V,masked", [(1, 1, 0), (3, 7, 0), (4, 1000, 0.5), (5, 16385, 0), (3, 50001, 0.25)])
@pytest.mark.parametrize("with_entropy", [True, False])
def test_logprobs_grad(M, V, masked, dt, with_entropy):
    x, t, lse, H, gl, gh = grad_case(M, V, dt, V + M, masked)
    if M > 3:
        x[0] = -math.inf
        lse[0], H[0] = -math.inf, 0.0
        t[0] = 0
    want, tol = logprobs_grad(x, t, lse, gl, H, gh if with_entropy else None, dt)
    got = om.token_logprobs_grad(x.cuda(), t.cuda(), lse.cuda(), gl.cuda(), H.cuda() if with_entropy else None,
                                 gh.cuda() if with_entropy else None)
    assert_within(got, want, tol)


def test_logprobs_grad_in_place_and_misaligned():
    x, t, lse, H, gl, gh = grad_case(3, 1003, "bf16", 11, 0.1)
    want, tol = logprobs_grad(x, t, lse, gl, H, gh, "bf16")
    args = (t.cuda(), lse.cuda(), gl.cuda(), H.cuda(), gh.cuda())
    y = x.cuda()
    om.token_logprobs_grad(y, *args, grad_logits=y)
    assert_within(y, want, tol, "in place")
    buf = torch.full((3 * 1003 + 9,), 7.0, dtype=torch.bfloat16, device="cuda")
    om.token_logprobs_grad(x.cuda(), *args, grad_logits=buf[5:5 + 3009].view(3, 1003))
    assert_within(buf[5:5 + 3009].view(3, 1003), want, tol, "misaligned")
    assert bool((buf[:5] == 7).all()) and bool((buf[-4:] == 7).all())


def test_logprobs_grad_against_differences():
    """Central differences of the 64-bit forward along random directions; the gradient is the GPU's fp32 one."""
    x, t, lse, H, gl, gh = grad_case(4, 200, "f32", 3)
    got = om.token_logprobs_grad(x.cuda(), t.cuda(), lse.cuda(), gl.cuda(), H.cuda(), gh.cuda()).double().cpu()

    def loss(z):
        (lp, ent, _, _, _), _ = logprobs(z, t, 0)
        return float((gl.double() * lp + gh.double() * ent).sum())

    gen = torch.Generator().manual_seed(4)
    h = 1e-5
    for _ in range(4):
        v = torch.randn(x.shape, generator=gen, dtype=torch.float64)
        num = (loss(x.double() + h * v) - loss(x.double() - h * v)) / (2 * h)
        # h^2 times the third derivative (order 10 |v|^3) plus the fp32 gradient's error
        assert abs(num - float((got * v).sum())) <= 1e-5


def test_logprobs_past_32_bit_offsets():
    M, V = 70000, 32768  # 2.3e9 elements
    x = torch.zeros((M, V), dtype=torch.bfloat16, device="cuda")
    last, t = rows(4, V, "bf16", 9)
    x[-4:] = last.cuda()
    targets = torch.zeros((M,), dtype=torch.int64)
    targets[-4:] = t
    got = om.token_logprobs(x, targets.cuda(), top_k=0)
    want, tol = logprobs(last, t, 0)
    for i in (0, 1, 2):
        assert_within(got[i][-4:], want[i], tol[i], str(i))
        assert bool((got[i][:5] == got[i][0]).all())
    gl, gh = torch.ones((M,)), torch.ones((M,))
    g = om.token_logprobs_grad(x, targets.cuda(), got[2], gl.cuda(), got[1], gh.cuda(), grad_logits=x)
    wg, tg = logprobs_grad(last, t, got[2][-4:].cpu(), gl[-4:], got[1][-4:].cpu(), gh[-4:], "bf16")
    assert_within(g[-4:], wg, tg)
