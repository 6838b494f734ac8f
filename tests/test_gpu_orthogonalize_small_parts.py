"""orthogonalize of a matrix whose parts differ in size by many orders: what the contract says of the small ones."""
import pytest
import torch

from tests.decode_util import TORCH, assert_within, half_step
from tests.train_util import COEFFICIENTS, orthogonalise

pytestmark = pytest.mark.gpu

om = pytest.importorskip("onnx_matmul_family_amd._omm")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    om.lib()


@pytest.mark.parametrize("tall", [False, True])
@pytest.mark.parametrize("size", [1e-6, 1e-7, 1e-8, 1e-9, 1e-10])
def test_small_block_beside_a_large_one(size, tall):
    """Blocks on the diagonal do not meet, and the small one's singular values stay so small that a step multiplies
    it by a = 3.4445 (B = a I to 1e-7).  An entry x is held to 2^-22 of itself, no finer than 2^-39 of |G| (half the
    smallest step of fp16, 2^-24, over the scale 2^14), at the start and after every step but the last; a step's
    product is off by 3 2^-22 of it (a in two parts, the two small parts' product, fp32 sums).  An error of one step
    is multiplied by a in each that follows."""
    gen = torch.Generator().manual_seed(7)
    big, small = torch.randn((48, 80), generator=gen), torch.randn((40, 64), generator=gen)
    big /= torch.linalg.vector_norm(big)
    G = torch.zeros((88, 144))
    G[:48, :80], G[48:, 80:] = big, small * size
    got = om.orthogonalize((G.t().contiguous() if tall else G).cuda())[0].cpu()
    got = got.t() if tall else got
    want = orthogonalise(G, 5)
    a = COEFFICIENTS[0]
    floor = sum(a ** (5 - i) for i in range(5)) * 2.0 ** -39
    tol = 1.01 * (floor + 21 * 2.0 ** -22 * want.abs())
    assert_within(got[48:, 80:], want[48:, 80:], (tol + half_step("f32", want.abs() + tol))[48:, 80:], "small block")
    assert (got[:48, 80:] == 0).all() and (got[48:, :80] == 0).all()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_entries_below_the_smallest_step(dt):
    """What is below 2^-40 of |G| may be 0: the rest is what it is without it."""
    gen = torch.Generator().manual_seed(8)
    G = torch.zeros((70, 100))
    G[:60, :90] = torch.randn((60, 90), generator=gen)
    G = G.to(TORCH[dt])
    H = G.clone()
    H[60:, 90:] = torch.randn((10, 10), generator=gen).to(TORCH[dt]) * 1e-16
    a, b = om.orthogonalize(G.cuda())[0], om.orthogonalize(H.cuda())[0]
    assert torch.equal(a[:60, :90], b[:60, :90]) and (b[60:, 90:] == 0).all()
