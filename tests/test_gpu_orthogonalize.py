"""orthogonalize against its definition in 64 bits."""
import math

import pytest
import torch

from tests.decode_util import TORCH, assert_within
from tests.train_util import orthogonalise, orthogonalise_tol

pytestmark = pytest.mark.gpu

om = pytest.importorskip("onnx_matmul_family_amd._omm")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    om.lib()


def draw(m, n, dt, rank=0, seed=0):
    gen = torch.Generator().manual_seed(seed)
    G = torch.randn((m, n), generator=gen) * 1e-3
    if rank:
        G = G + torch.randn((m, rank), generator=gen) @ torch.randn((rank, n), generator=gen) * 1e-2
    return G.to(TORCH[dt])


def check(G, got, steps, dt):
    want = orthogonalise(G, steps)
    assert_within(got, want, orthogonalise_tol(G, want, steps, dt), "%s x %s" % tuple(G.shape))


SIZES = [(1, 1), (1, 7), (9, 1), (2, 3), (16, 16), (31, 65), (64, 64), (100, 40), (127, 129), (128, 128), (130, 128),
         (128, 130), (200, 333), (333, 200), (257, 64), (64, 500), (256, 256), (300, 300)]


@pytest.mark.parametrize("m,n", SIZES)
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_sizes(m, n, dt):
    G = draw(m, n, dt, seed=m + n)
    got, ws = om.orthogonalize(G.cuda())
    assert got.dtype == G.dtype and ws.dtype == torch.uint8
    check(G, got, 5, dt)


@pytest.mark.parametrize("Z,m,n,dt", [(1, 4096, 4096, "f32"), (1, 2100, 3300, "bf16"), (6, 1000, 1024, "f32"),
                                      (16, 1024, 1000, "bf16"), (1, 1500, 700, "f16")])
def test_large(Z, m, n, dt):
    """The larger tiles.  The definition on the GPU here, in 64 bits, by library products."""
    G = torch.stack([draw(m, n, dt, rank=4, seed=z) for z in range(Z)]).cuda()
    got, _ = om.orthogonalize(G)
    for z in {0, Z - 1}:
        want = orthogonalise(G[z], 5)
        tol = orthogonalise_tol(G[z], want, 5, dt)
        assert_within(got[z], want.cpu(), tol.cpu(), "%d of %d" % (z, Z))


@pytest.mark.parametrize("steps", [1, 2, 3, 8])
@pytest.mark.parametrize("m,n", [(60, 90), (150, 70)])
def test_steps(m, n, steps):
    G = draw(m, n, "f32")
    check(G, om.orthogonalize(G.cuda(), steps=steps)[0], steps, "f32")


@pytest.mark.parametrize("m,n,rank", [(200, 300, 4), (300, 160, 16)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_few_directions_stand_out(m, n, rank, dt):
    G = draw(m, n, dt, rank)
    check(G, om.orthogonalize(G.cuda())[0], 5, dt)


@pytest.mark.parametrize("Z,m,n", [(1, 20, 30), (3, 140, 90), (5, 64, 200), (17, 33, 33)])
def test_batches(Z, m, n):
    """Each matrix as if it were alone, whatever the others hold."""
    G = torch.stack([draw(m, n, "f32", seed=z) * 10.0 ** (z % 5 - 2) for z in range(Z)])
    got, _ = om.orthogonalize(G.cuda())
    for z in range(Z):
        check(G[z], got[z], 5, "f32")
        assert torch.equal(got[z], om.orthogonalize(G[z].cuda())[0])
    if Z > 2:
        G[0, 3, 5], G[1] = math.nan, 0
        G[2, 0, 0] = math.inf
        again, _ = om.orthogonalize(G.cuda())
        assert again[0].isnan().all() and (again[1] == 0).all() and again[2].isnan().all()
        assert torch.equal(again[3:], got[3:])


@pytest.mark.parametrize("scale", [1e-38, 1e-42, 1e-20, 1e18, 1e37])
def test_size_of_the_matrix_does_not_matter(scale):
    """fp32 squares of these would be 0 or infinite (of 1e-42 the entries have few bits: the oracle reads the same)."""
    G = (draw(40, 70, "f32") * 1e3).double().mul(scale).float()
    check(G, om.orthogonalize(G.cuda())[0], 5, "f32")


def test_diagonal_and_signs():
    """Entries of 1 in the normalised matrix; a matrix of one entry."""
    G = torch.zeros((50, 60))
    G[7, 9] = -3.0
    got, _ = om.orthogonalize(G.cuda())
    check(G, got, 5, "f32")
    D = torch.diag(torch.linspace(-1, 1, 40))
    check(D, om.orthogonalize(D.cuda())[0], 5, "f32")


def test_singular_values():
    """What it is for: they come near 1, the singular vectors stay."""
    G = draw(96, 160, "f32")
    X = om.orthogonalize(G.cuda())[0].double().cpu()
    s = torch.linalg.svdvals(X)
    assert float(s.max()) < 1.3 and float(s.min()) > 0.5
    U, _, V = torch.linalg.svd(G.double(), full_matrices=False)
    off = U.t() @ X @ V.t()
    assert float((off - torch.diag(torch.diag(off))).abs().max()) < 1e-4


def test_in_place_and_given_buffers():
    G = draw(77, 130, "bf16").cuda()
    want, _ = om.orthogonalize(G)
    ws = torch.full((om.orthogonalize_workspace_size(1, 77, 130),), 255, dtype=torch.uint8, device="cuda")
    H = G.clone()
    out, w = om.orthogonalize(H, out=H, workspace=ws)
    assert out.data_ptr() == H.data_ptr() and w.data_ptr() == ws.data_ptr()
    assert torch.equal(out, want)


@pytest.mark.parametrize("Z,m,n", [(1, 37, 51), (2, 129, 40)])
def test_nothing_outside(Z, m, n):
    G = torch.stack([draw(m, n, "f32", seed=z) for z in range(Z)])
    y = torch.full((Z * m * n + 512,), 7.0, device="cuda")
    need = om.orthogonalize_workspace_size(Z, m, n)
    ws = torch.full((need + 512,), 77, dtype=torch.uint8, device="cuda")
    om.orthogonalize(G.cuda(), out=y[256:256 + Z * m * n].view(Z, m, n), workspace=ws[256:256 + need])
    assert (y[:256] == 7).all() and (y[256 + Z * m * n:] == 7).all()
    assert (ws[:256] == 77).all() and (ws[256 + need:] == 77).all()


def test_unaligned_input():
    pool = torch.zeros((90 * 61 + 8,), dtype=torch.bfloat16, device="cuda")
    G = draw(90, 61, "bf16")
    pool[3:3 + 90 * 61] = G.cuda().reshape(-1)
    check(G, om.orthogonalize(pool[3:3 + 90 * 61].view(90, 61))[0], 5, "bf16")


def test_empty():
    assert om.orthogonalize(torch.empty((0, 5), device="cuda"))[0].shape == (0, 5)
    assert om.orthogonalize(torch.empty((2, 5, 0), device="cuda"))[0].shape == (2, 5, 0)


@pytest.mark.parametrize("Z,m,n,dt", [(1, 40, 4000, "f32"), (1, 64, 2496, "bf16"), (3, 128, 2500, "f32"), (18, 3200, 192, "bf16"),
                                      (5, 1, 900, "f32"), (1, 4096, 96, "f16"), (1, 33, 513, "f32")])
def test_long(Z, m, n, dt):
    """Few tiles and a long contraction, in order and again: the same bits, whatever the workspace held."""
    G = torch.stack([draw(m, n, dt, rank=2, seed=z) for z in range(Z)])
    size = om.orthogonalize_workspace_size(Z, m, n)
    first = None
    for fill in (0, 255):
        ws = torch.full((size,), fill, dtype=torch.uint8, device="cuda")
        got, _ = om.orthogonalize(G.cuda(), workspace=ws)
        for z in range(Z):
            check(G[z], got[z], 5, dt)
        again, _ = om.orthogonalize(G.cuda(), workspace=ws)
        first = got if first is None else first
        assert torch.equal(got, first) and torch.equal(again, first)


def test_long_in_a_graph():
    """Replays with new inputs, eager calls on the same workspace between them."""
    G = torch.stack([draw(96, 2000, "f32", rank=3, seed=z) for z in range(5)]).cuda()
    ws = torch.empty((om.orthogonalize_workspace_size(1, 96, 2000),), dtype=torch.uint8, device="cuda")
    src, out = G[0].clone(), torch.empty_like(G[0])
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        om.orthogonalize(src, out=out, workspace=ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            om.orthogonalize(src, out=out, workspace=ws)
    for z in range(1, 5):
        src.copy_(G[z])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        eager, _ = om.orthogonalize(G[z], workspace=ws)
        torch.cuda.synchronize()
        assert torch.equal(got, eager)
        check(G[z].cpu(), got, 5, "f32")
