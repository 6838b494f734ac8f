"""lora_matmul rounds the whole sum once, but where include/omm.h says otherwise (tests/decode_util.py's bound
without the room for a second rounding), and a row's bits do not depend on the others."""
import pytest
import torch

from tests.decode_util import TORCH, assert_within, half_step, lora
from tests.test_gpu_lora import case as lora_case, run as run_lora

pytestmark = pytest.mark.gpu

om = pytest.importorskip("onnx_matmul_family_amd._omm")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    om.lib()


def cancelling(M, K, N, R, G, dt, trans, big, seed):
    """X W = -2 big + .., the adapter's term 2 big + ..: what rounds or overflows alone shows in the sum."""
    X, W, A, B, _, _, _ = lora_case(M, K, N, R, G, dt, trans, seed, bias=False, scale=False)
    idx = torch.arange(M) % G
    X[:, :2] = 1.0
    if trans:
        W, A, B = W.t(), A.transpose(1, 2), B.transpose(1, 2)
    W[:2] = -big
    A[:, :2] = 0.0
    A[:, 0, 0] = A[:, 1, 1] = 1.0
    A[:, 2:, :2] = 0.0
    B[:, :2] = big
    if trans:
        W, A, B = W.t().contiguous(), A.transpose(1, 2).contiguous(), B.transpose(1, 2).contiguous()
    return X, W, A, B, idx, None, None


def once(c, trans, dt):
    """(Y, bound with one rounding)."""
    want, tol = lora(*c, trans, dt)
    term, _ = lora(c[0], c[1] * 0, *c[2:], trans, dt)
    return want, tol - half_step(dt, term)


def check(c, trans, dt, sel=None):
    got, _ = run_lora(c, trans)
    if sel is not None:
        c = (c[0][sel], c[1], c[2], c[3], c[4][sel], c[5], c[6])
        got = got[sel.cuda()]
    want, tol = once(c, trans, dt)
    assert_within(got, want, tol)


@pytest.mark.parametrize("dt,big", [("bf16", 4.0), ("f16", 4.0), ("f16", 40000.0)])
@pytest.mark.parametrize("trans", [0, 1])
@pytest.mark.parametrize("M,K,N,R,G", [(1, 64, 64, 8, 1), (43, 520, 136, 24, 5), (300, 136, 264, 16, 3),
                                       (700, 128, 264, 16, 3), (1024, 64, 16384, 16, 3), (700, 129, 267, 16, 3),
                                       (300, 128, 264, 4, 3), (700, 128, 264, 4, 3)])
def test_one_rounding(M, K, N, R, G, dt, big, trans):
    check(cancelling(M, K, N, R, G, dt, trans, big, M + K), trans, dt)


@pytest.mark.parametrize("dt,big", [("bf16", 4.0), ("f16", 40000.0)])
@pytest.mark.parametrize("trans", [0, 1])
@pytest.mark.parametrize("M,K,N,R,G", [(65536, 33, 41, 9, 5), (66001, 33, 41, 9, 5), (66001, 64, 72, 4, 5),
                                       (131073, 41, 33, 2, 3)])
def test_one_rounding_of_65536_rows_and_more(M, K, N, R, G, dt, big, trans):
    sel = torch.cat([torch.arange(0, M, 997), torch.arange(max(0, M - 70), M)]).unique()
    check(cancelling(M, K, N, R, G, dt, trans, big, M), trans, dt, sel)


@pytest.mark.parametrize("trans", [0, 1])
def test_one_rounding_of_an_x_of_2_gib(trans):
    """262144 + 3 rows of 4096: past 32-bit byte offsets into X."""
    M, K, N, R, G = 262147, 4096, 64, 8, 3
    c = list(cancelling(8, K, N, R, G, "bf16", trans, 4.0, 5))
    gen = torch.Generator(device="cuda").manual_seed(6)
    X = torch.randn((M, K), generator=gen, device="cuda", dtype=torch.bfloat16)
    X[:, :2] = 1.0
    idx = torch.arange(M) % G
    got, _ = om.lora_matmul(X, *[t.cuda() for t in c[1:4]], idx.cuda(), trans=trans)
    sel = torch.cat([torch.arange(0, M, 9973), torch.tensor([131071, 131072, 262143, 262144, M - 1])]).unique()
    c[0], c[4] = X[sel.cuda()].cpu(), idx[sel]
    want, tol = once(c, trans, "bf16")
    assert_within(got[sel.cuda()], want, tol)


@pytest.mark.parametrize("trans", [0, 1])
@pytest.mark.parametrize("M", [20, 40, 300, 600, 1100])
def test_bits_of_a_row_do_not_depend_on_other_rows_adapters(M, trans):
    """Also inside blocks of 16 rows that mix adapters."""
    c = [t.cuda() for t in lora_case(M, 256, 520, 16, 8, "bf16", trans, 71)]
    a, _ = om.lora_matmul(*c, trans=trans)
    keep = torch.arange(M, device="cuda") % 3 == 0
    for step in (1, 3):
        other = list(c)
        other[4] = torch.where(keep, c[4], (c[4] + 1 + step) % 9 - 1)
        b, _ = om.lora_matmul(*other, trans=trans)
        assert torch.equal(a[keep].view(torch.int16), b[keep].view(torch.int16))
        assert not torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("dt", ["bf16", "f16"])
@pytest.mark.parametrize("trans", [0, 1])
def test_w_of_2_gib(dt, trans):
    """No multiples of 8: the one 16-bit form besides the element-wise one that may round the term first."""
    M, K, N, R, G = 70, 32769, 32771, 9, 3
    gen = torch.Generator(device="cuda").manual_seed(7)

    def make(*shape, std):
        return torch.randn(shape, generator=gen, device="cuda", dtype=TORCH[dt]) * std

    X, W = make(M, K, std=1.0), make(*((N, K) if trans else (K, N)), std=K ** -0.5)
    A, B = make(*((G, R, K) if trans else (G, K, R)), std=K ** -0.5), make(*((G, N, R) if trans else (G, R, N)), std=0.3)
    bias, idx = make(N, std=0.5), torch.arange(M) % (G + 1) - 1
    got, _ = om.lora_matmul(X, W, A, B, idx.cuda(), None, bias, trans=trans)
    cols = torch.cat([torch.arange(40), torch.arange(N // 2, N // 2 + 40), torch.arange(N - 40, N)]).cuda()
    dim = 0 if trans else 1
    want, tol = lora(X.cpu(), W.index_select(dim, cols).cpu(), A.cpu(), B.index_select(dim + 1, cols).cpu(), idx, None,
                     bias[cols].cpu(), trans, dt)
    assert_within(got[:, cols], want, tol)


@pytest.mark.parametrize("trans", [0, 1])
def test_element_wise_form_in_pieces(trans):
    """4 deep, 2^22 columns and more: 1023 rows a launch."""
    M, K, N, R, G = 1100, 4, (1 << 22) + 5, 2, 3
    gen = torch.Generator(device="cuda").manual_seed(8)

    def make(*shape):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16)

    X, W = make(M, K), make(*((N, K) if trans else (K, N)))
    A, B = make(*((G, R, K) if trans else (G, K, R))), make(*((G, N, R) if trans else (G, R, N)))
    idx = torch.arange(M) % (G + 1) - 1
    got, _ = om.lora_matmul(X, W, A, B, idx.cuda(), trans=trans)
    cols = torch.cat([torch.arange(40), torch.arange(N // 2, N // 2 + 40), torch.arange(N - 40, N)]).cuda()
    dim = 0 if trans else 1
    want, tol = lora(X.cpu(), W.index_select(dim, cols).cpu(), A.cpu(), B.index_select(dim + 1, cols).cpu(), idx, None,
                     None, trans, "bf16")
    assert_within(got[:, cols], want, tol)
