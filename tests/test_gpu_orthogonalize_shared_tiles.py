"""orthogonalize where several workgroups share a tile's contraction and meet in the workspace: its bounds and
contents, calls that overlap, two graphs on one workspace."""
import pytest
import torch

from tests.test_gpu_decode_workspaces import within

pytestmark = pytest.mark.gpu

om = pytest.importorskip("onnx_matmul_family_amd._omm")

SHAPES = [(1, 96, 2000), (1, 64, 2496), (1, 320, 5000), (1, 1440, 720), (3, 128, 2500), (18, 3200, 192), (1, 4096, 96)]


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    om.lib()


def matrix(Z, m, n, seed=0):
    gen = torch.Generator(device="cuda").manual_seed(seed + m)
    return torch.randn((Z, m, n), generator=gen, device="cuda")


@pytest.mark.parametrize("Z,m,n", SHAPES)
def test_workspace(Z, m, n):
    G = matrix(Z, m, n)
    within(om.orthogonalize_workspace_size(Z, m, n), lambda ws: om.orthogonalize(G, workspace=ws)[:1])


def test_calls_that_overlap():
    """On four streams, with workspaces of their own."""
    Gs = [matrix(*s, seed=i) for i, s in enumerate(SHAPES)]
    want = [om.orthogonalize(G)[0].clone() for G in Gs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for r in range(4):
        for i, G in enumerate(Gs):
            got.append((i, om.orthogonalize(G, stream=streams[(i + r) % 4])[0]))
    torch.cuda.synchronize()
    for i, g in got:
        assert torch.equal(g, want[i]), SHAPES[i]


@pytest.mark.parametrize("Z,m,n", [(3, 128, 2500), (18, 3200, 192)])
def test_a_matrix_that_is_not_finite(Z, m, n):
    """NaN and zeros in a batch stay in their matrices, and in the call that they came with."""
    G = matrix(Z, m, n)
    ws = torch.empty((om.orthogonalize_workspace_size(Z, m, n),), dtype=torch.uint8, device="cuda")
    want = om.orthogonalize(G, workspace=ws)[0].clone()
    bad = G.clone()
    bad[0, 5, 7], bad[1] = float("nan"), 0.0
    bad[2, m - 1, n - 1] = float("inf")
    got = om.orthogonalize(bad, workspace=ws)[0]
    assert got[0].isnan().all() and (got[1] == 0).all() and got[2].isnan().all() and torch.equal(got[3:], want[3:])
    assert torch.equal(om.orthogonalize(G, workspace=ws)[0], want)


def test_two_graphs_on_one_workspace():
    """One after the other, over what the other one left."""
    shapes = [(1, 96, 2000), (18, 3200, 192)]
    ws = torch.full((max(om.orthogonalize_workspace_size(*s) for s in shapes),), 255, dtype=torch.uint8, device="cuda")
    Gs = [[matrix(*s, seed=k) for k in range(3)] for s in shapes]
    want = [[om.orthogonalize(G)[0].clone() for G in g] for g in Gs]
    graphs = []
    for g in Gs:
        src, out = g[0].clone(), torch.empty_like(g[0])
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            om.orthogonalize(src, out=out, workspace=ws)
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                om.orthogonalize(src, out=out, workspace=ws)
        graphs.append((graph, src, out))
    for r in range(6):
        i, k = r % 2, r % 3
        graph, src, out = graphs[i]
        src.copy_(Gs[i][k])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i][k])
