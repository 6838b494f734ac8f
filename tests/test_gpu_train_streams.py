"""The operators that train, balance and quantise: workspaces, other streams, graphs, long offsets, refusals
of the binding."""
import pytest
import torch

from tests.decode_util import TORCH
from tests.test_gpu_decode_workspaces import within

pytestmark = pytest.mark.gpu

om = pytest.importorskip("onnx_matmul_family_amd._omm")

WAIT = 40_000_000  # clock ticks that keep a stream busy while the host goes on (20 ms or so)


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    om.lib()


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def product_case(M, K, N, dt="bf16"):
    X = torch.randn((M, K), generator=gen(M), device="cuda").to(TORCH[dt])
    W, s = om.quantize_rows(torch.randn((N, K), generator=gen(N), device="cuda"))
    return X, W, s


def router_case(M, E, k):
    x = torch.randn((M, E), generator=gen(M), device="cuda")
    return x, torch.topk(x, k, dim=1)[1].to(torch.int32)


# ---------------------------------------------------------------- workspaces

@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,K,N", [(1, 4096, 100), (5, 333, 70), (40, 1000, 130), (100, 256, 128), (300, 2005, 200),
                                   (70, 31, 9000), (520, 1024, 520)])
def test_product_workspace(M, K, N, dt):
    X, W, s = product_case(M, K, N, dt)
    within(om.int8_matmul_workspace_size(M, K, N, TORCH[dt]), lambda ws: om.int8_matmul(X, W, s, workspace=ws)[:1])
    q, qs = om.quantize_rows(X)
    within(om.int8_matmul_workspace_size(M, K, N, torch.int8),
           lambda ws: om.int8_matmul(q, W, s, a_scale=qs, workspace=ws if ws.numel() else None)[:1])


@pytest.mark.parametrize("M,E,k", [(300, 64, 4), (1000, 60, 8), (20000, 512, 16), (9000, 130, 1)])
def test_balance_workspace(M, E, k):
    x, ids = router_case(M, E, k)
    within(om.moe_balance_workspace_size(M, E), lambda ws: om.moe_balance(x, ids, workspace=ws))


@pytest.mark.parametrize("Z,m,n", [(1, 5, 7), (1, 300, 500), (3, 257, 129), (4, 640, 1000), (1, 2000, 1100)])
def test_orthogonalize_workspace(Z, m, n):
    G = torch.randn((Z, m, n), generator=gen(m), device="cuda")
    within(om.orthogonalize_workspace_size(Z, m, n), lambda ws: om.orthogonalize(G, workspace=ws)[:1])


# ---------------------------------------------------------------- streams

def calls():
    X, W, s = product_case(300, 512, 520)
    odd = product_case(200, 333, 260)
    few = product_case(1, 4096, 1000)
    x, ids = router_case(5000, 64, 4)
    _, counts, tokens = om.moe_balance(x, ids)
    g, gl = torch.randn((5000, 4), generator=gen(1), device="cuda"), torch.ones((2,), device="cuda")
    G = torch.randn((200, 300), generator=gen(2), device="cuda")
    return {
        "quantize": lambda st: om.quantize_rows(X, stream=st),
        "product": lambda st: om.int8_matmul(X, W, s, stream=st)[:1],
        "odd": lambda st: om.int8_matmul(*odd, stream=st)[:1],
        "few": lambda st: om.int8_matmul(*few, stream=st)[:1],
        "balance": lambda st: om.moe_balance(x, ids, stream=st),
        "grad": lambda st: (om.moe_route_grad(x, ids, g, counts=counts, tokens=tokens, grad_losses=gl, stream=st),),
        "orthogonalize": lambda st: om.orthogonalize(G, stream=st)[:1],
    }


NAMES = ["quantize", "product", "odd", "few", "balance", "grad", "orthogonalize"]


@pytest.mark.parametrize("name", NAMES)
def test_on_another_stream(name):
    """The stream is busy, so the call's kernels run after these tensors were made and filled."""
    call = calls()[name]
    want = [t.clone() for t in call(None)]
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(WAIT)
    got = call(s)
    mine = [torch.full((1 << 20,), 77, dtype=torch.uint8, device="cuda") for _ in range(6)]
    torch.cuda.current_stream().synchronize()
    s.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for t in mine:
        assert bool((t == 77).all())


def test_two_streams_at_once():
    """Calls that overlap share nothing."""
    cs = calls()
    want = {n: [t.clone() for t in c(None)] for n, c in cs.items()}
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(4)]
    got = []
    for r in range(3):
        for i, n in enumerate(NAMES):
            got.append((n, cs[n](streams[(i + r) % 4])))
    torch.cuda.synchronize()
    for n, out in got:
        for a, b in zip(out, want[n]):
            assert torch.equal(a, b), n


# ---------------------------------------------------------------- graphs

@pytest.mark.parametrize("name", NAMES)
def test_captured_and_replayed(name):
    """Replays with other inputs in the captured buffers, eager work between them; two graphs alive at once."""
    Xs = [product_case(300, 512, 520)[0] * k for k in (1, 2, 3)]
    few = [product_case(1, 4096, 1000)[0] * k for k in (1, 2, 3)]
    odd = [product_case(200, 333, 260)[0] * k for k in (1, 2, 3)]
    xs = [router_case(5000, 64, 4)[0] * k for k in (1, 2, 3)]
    Gs = [torch.randn((200, 300), generator=gen(k), device="cuda") for k in (1, 2, 3)]
    _, W, s = product_case(300, 512, 520)
    _, Wf, sf = product_case(1, 4096, 1000)
    _, Wo, so = product_case(200, 333, 260)
    ids = router_case(5000, 64, 4)[1]
    gw = torch.randn((5000, 4), generator=gen(1), device="cuda")

    def grad(x):
        losses, counts, tokens = om.moe_balance(x, ids)
        return (om.moe_route_grad(x, ids, gw, counts=counts, tokens=tokens, grad_losses=losses),)

    inputs, f = {"quantize": (Xs, om.quantize_rows), "product": (Xs, lambda x: om.int8_matmul(x, W, s)[:1]),
                 "few": (few, lambda x: om.int8_matmul(x, Wf, sf)[:1]), "odd": (odd, lambda x: om.int8_matmul(x, Wo, so)[:1]),
                 "balance": (xs, lambda x: om.moe_balance(x, ids)), "grad": (xs, grad),
                 "orthogonalize": (Gs, lambda x: om.orthogonalize(x)[:1])}[name]
    want = [[t.clone() for t in f(x)] for x in inputs]
    graphs = []
    for _ in range(2):
        buf = inputs[0].clone()
        st = torch.cuda.Stream()
        st.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(st):
            f(buf)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            out = f(buf)
        graphs.append((g, buf, out))
    for r in range(4):
        for i, (g, buf, out) in enumerate(graphs):
            k = (r + i) % 3
            buf.copy_(inputs[k])
            g.replay()
            eager = f(inputs[(k + 1) % 3])
            torch.cuda.synchronize()
            for a, b in zip(out, want[k]):
                assert torch.equal(a, b)
            for a, b in zip(eager, want[(k + 1) % 3]):
                assert torch.equal(a, b)


# ---------------------------------------------------------------- long offsets

@pytest.mark.parametrize("M,K", [(1, 4096), (40, 4096), (130, 4096), (3, 4099)])
def test_weights_past_32_bits(M, K):
    """More than 2^32 bytes of weights: columns at the end come out as by themselves."""
    N = 2 ** 32 // K + 5000
    W = torch.randint(-128, 128, (N, K), generator=gen(0), device="cuda", dtype=torch.int8)
    sb = torch.rand((N,), generator=gen(1), device="cuda")
    X = torch.randn((M, K), generator=gen(2), device="cuda").to(torch.bfloat16)
    Y, _ = om.int8_matmul(X, W, sb)
    for lo in (0, 2 ** 31 // K - 50, N - 300):
        part, _ = om.int8_matmul(X, W[lo:lo + 300].clone(), sb[lo:lo + 300].clone())
        assert torch.equal(Y[:, lo:lo + 300], part)


def test_rows_past_32_bits():
    M, K = 2 ** 32 // 8192 + 700, 8192
    X = torch.empty((M, K), device="cuda", dtype=torch.bfloat16).normal_(generator=gen(0))
    q, s = om.quantize_rows(X)
    W, sb = om.quantize_rows(torch.randn((64, K), generator=gen(3), device="cuda"))
    Y, _ = om.int8_matmul(q, W, sb, a_scale=s)
    for lo in (0, 2 ** 31 // K - 5, M - 300):
        qq, ss = om.quantize_rows(X[lo:lo + 300].clone())
        assert torch.equal(q[lo:lo + 300], qq) and torch.equal(s[lo:lo + 300], ss)
        assert torch.equal(Y[lo:lo + 300], om.int8_matmul(qq, W, sb, a_scale=ss)[0])


def test_logits_past_32_bits():
    M, E = 2 ** 32 // 512 + 900, 512
    x = torch.empty((M, E), device="cuda", dtype=torch.bfloat16).normal_(generator=gen(0))
    ids = torch.randint(0, E, (M, 2), generator=gen(1), device="cuda", dtype=torch.int32)
    mask = torch.zeros((M,), dtype=torch.bool, device="cuda")
    mask[-300:] = True
    a = om.moe_balance(x, ids, token_mask=mask)
    b = om.moe_balance(x[-300:].clone(), ids[-300:].clone())
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    assert torch.allclose(a[0], b[0], rtol=300 * 2.0 ** -24)  # (300 terms, in another order)
    g = torch.randn((M, 2), generator=gen(2), device="cuda")
    d = om.moe_route_grad(x, ids, g, counts=a[1], tokens=a[2], grad_losses=a[0])
    for lo in (0, 2 ** 31 // E - 50, M - 300):
        part = om.moe_route_grad(x[lo:lo + 300].clone(), ids[lo:lo + 300].clone(), g[lo:lo + 300].clone(), counts=a[1],
                                 tokens=a[2], grad_losses=a[0])
        assert torch.equal(d[lo:lo + 300], part)


# ---------------------------------------------------------------- refusals of the binding

def test_refusals():
    X, W, s = product_case(4, 32, 8)
    x, ids = router_case(6, 8, 2)

    def code(f, *a, **kw):
        with pytest.raises(om.OmmError) as e:
            f(*a, **kw)
        return e.value.code

    assert code(om.int8_matmul, X, W, s[:7].contiguous()) == -3
    assert code(om.int8_matmul, X.double(), W, s, dtype=torch.bfloat16) == -5
    assert code(om.int8_matmul, W, W, s) == -1  # an int8 a without its scales
    assert code(om.int8_matmul, X, W, s, a_scale=s) == -3
    assert code(om.int8_matmul, X, W, s, bias=s) == -2
    assert code(om.int8_matmul, X, W, s, workspace=torch.empty((64,), dtype=torch.uint8, device="cuda")) == -6
    assert code(om.quantize_rows, X.to(torch.int32)) == -2
    assert code(om.moe_balance, x, ids, token_mask=x[:, 0].contiguous()) == -2
    assert code(om.moe_balance, x, ids.float()) == -2
    assert code(om.moe_route_grad, x, ids, grad_losses=x[0, :2].contiguous()) == -1
    assert code(om.orthogonalize, x, steps=0) == -5
    assert code(om.orthogonalize, x.double()) == -5
    assert code(om.orthogonalize, x, out=x[:5].contiguous()) == -3
    for f, args in ((om.int8_matmul, (X.cpu(), W, s)), (om.int8_matmul, (X, W.cpu(), s)), (om.int8_matmul, (X, W.t(), s)),
                    (om.int8_matmul, (X[0], W, s)), (om.quantize_rows, (X.t(),)), (om.moe_balance, (x, ids.cpu())),
                    (om.moe_balance, (x[0], ids)), (om.orthogonalize, (x.t(),)), (om.orthogonalize, (x[0],))):
        with pytest.raises(ValueError):
            f(*args)
    with pytest.raises(ValueError):
        om.int8_matmul(X, W, s, dtype=torch.float64)
    assert code(om.int8_matmul, X, W, None) == -1
    with pytest.raises(OverflowError):
        om.orthogonalize(x, steps=2 ** 32 + 5)
