"""The decode-side operators on the GPU where their kernels change form or can go
wrong: row counts on both sides of each form's limit, many adapters, non-finite
values beside finite ones, rows whose largest logits share a thread, graph
replays.  Bounds from tests/decode_util.py."""
import math

import pytest
import torch

from tests.decode_util import TORCH, assert_within, draw, logprobs, logprobs_grad, lora, moe, route
from tests.test_gpu_logprobs import check as check_logprobs
from tests.test_gpu_lora import case as lora_case, check as check_lora, run as run_lora
from tests.test_gpu_moe import check_layer, layer_case

pytestmark = pytest.mark.gpu

om = pytest.importorskip("onnx_matmul_family_amd._omm")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    om.lib()


# ---------------------------------------------------------------- adapters

@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("trans", [0, 1])
@pytest.mark.parametrize("M,K,N,R,G", [
    (256, 264, 520, 16, 5), (257, 264, 520, 16, 5), (513, 512, 520, 33, 9), (700, 136, 264, 64, 3), (600, 128, 136, 4, 6),
    (530, 72, 264, 100, 4), (520, 4104, 24, 8, 2), (300, 101, 139, 17, 3), (1030, 33, 57, 9, 40), (18, 1025, 2309, 16, 4),
    (3, 600, 4999, 7, 2), (40, 513, 1100, 12, 33)])
def test_lora_forms(M, K, N, R, G, dt, trans):
    check_lora(lora_case(M, K, N, R, G, dt, trans, M + N + R, bias=bool(M % 2), runs=bool(G % 2)), trans, dt)


@pytest.mark.parametrize("trans", [0, 1])
def test_lora_whole_tiles(trans):
    """256 x 256 tiles (at least 256 of them), whole and with ragged edges; ranks over one and two steps of 32."""
    for M, N, R in ((1024, 16384, 16), (1000, 16520, 40), (1024, 16384, 72)):
        c = lora_case(M, 64, N, R, 3, "bf16", trans, R)
        check_lora(c, trans, "bf16")


@pytest.mark.parametrize("M", [9, 600])
def test_lora_more_adapters_than_sorted(M):
    check_lora(lora_case(M, 64, 72, 8, 1500, "bf16", 1, M), 1, "bf16")
    check_lora(lora_case(M, 64, 72, 8, 1023, "f16", 0, M), 0, "f16")


@pytest.mark.parametrize("trans", [0, 1])
@pytest.mark.parametrize("M", [30, 200, 800])
def test_lora_infinities_stay_in_their_adapters_rows(M, trans):
    """Mixed rows: an adapter of infinities and NaN beside finite ones."""
    c = lora_case(M, 128, 264, 16, 4, "bf16", trans, 50)
    want, tol = lora(*c, trans, "bf16")
    c[2][1, 0] = math.inf
    c[3][1, 0] = math.nan
    got, _ = run_lora(c, trans)
    keep = c[4] != 1
    assert_within(got[keep.cuda()], want[keep], tol[keep])


@pytest.mark.parametrize("M", [5, 300, 800])
def test_lora_middle_values_beyond_fp16(M):
    """X A up to 1e6 and down to 1e-6 in fp16 rows, brought back by B."""
    X, W, A, B, idx, s, b = lora_case(M, 256, 136, 16, 3, "f16", 1, 60)
    X[::2] *= 64
    A = A * 512
    A[1] = A[1] * 2.0 ** -18
    B[0], B[2] = B[0] * 2.0 ** -12, B[2] * 2.0 ** -12
    W = W * 2.0 ** -4
    check_lora((X, W, A, B, idx, s, b), 1, "f16")


@pytest.mark.parametrize("M", [40, 300, 600])
def test_lora_results_do_not_depend_on_other_rows(M):
    """The same row gives the same bits among other rows' adapters (same call size)."""
    c = [t.cuda() for t in lora_case(M, 256, 520, 16, 8, "bf16", 0, 70)]
    a, _ = om.lora_matmul(*c)
    other = list(c)
    other[4] = c[4].clone()
    other[4][1:] = (c[4][1:] + 3) % 8
    b, _ = om.lora_matmul(*other)
    assert_within(a[:1], b[:1].double().cpu(), 2.0 ** -8 * b[:1].double().cpu().abs() + 1e-6)
    a2, _ = om.lora_matmul(*c)
    assert torch.equal(a.view(torch.int16), a2.view(torch.int16))


# ---------------------------------------------------------------- experts

@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("trans", [0, 1])
@pytest.mark.parametrize("M,K,F,E,k", [(2, 1031, 517, 12, 3), (64, 129, 67, 3, 3), (1, 9, 8, 2, 2), (30, 520, 1001, 16, 4),
                                       (5, 77, 1500, 60, 6), (1, 3000, 12, 4, 1)])
def test_layer_odd_sizes(M, K, F, E, k, dt, trans):
    c = layer_case(M, K, F, E, k, dt, trans, M + F)
    check_layer(c[0], c[1], k, *c[2:], dt, trans, renorm=bool(F % 2), activation="gelu" if M % 2 else "silu")


def test_layer_nan_token_stays_alone():
    c = layer_case(20, 256, 192, 6, 2, "bf16", 0, 3)
    X, logits, Wg, Wu, Wd = c
    want, tol = moe(X, logits, 2, Wg, Wu, Wd, True, "silu", 0, "bf16")
    X[4] = math.nan
    got, _ = om.moe_layer(X.cuda(), logits.cuda(), 2, Wg.cuda(), Wu.cuda(), Wd.cuda())
    keep = torch.arange(20) != 4
    assert_within(got[keep.cuda()], want[keep], tol[keep])
    assert bool(got[4].isnan().all())


# ---------------------------------------------------------------- log probabilities

@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("V", [16384, 50001])
def test_logprobs_largest_logits_in_few_threads(V, dt):
    """The largest values next to each other, a thread's stride apart, and a whole row in bands."""
    gen = torch.Generator().manual_seed(V)
    x = torch.randn((6, V), generator=gen)
    x[0, 100:140] += 20 + torch.arange(40) / 8
    for stride in (2048, 1024):
        i = torch.arange(7, V, stride)[:40]
        x[1 if stride == 2048 else 2, i] += 30 - torch.arange(len(i)) / 4
    x[3] = (torch.arange(V) % 97) / 8.0
    x[4] = torch.where(torch.arange(V) < 40, torch.full((V,), 5.0), torch.full((V,), -5.0))
    x[5, ::2048] = 9.0
    t = torch.tensor([100, 7, 7, 96, 39, 0])
    for k in (1, 8, 32):
        check_logprobs(x.to(TORCH[dt]), t, k, "k=%d" % k)


@pytest.mark.parametrize("M", [1, 40, 600])
def test_logprobs_fewer_finite_than_wanted(M):
    """A grammar that leaves three tokens, of the lowest value and of -inf elsewhere."""
    V = 9000
    x = torch.full((M, V), -math.inf)
    x[:, [5, 4000, 8999]] = torch.tensor([1.0, 3.0, 2.0])
    t = torch.full((M,), 4000)
    check_logprobs(x, t, 8)
    check_logprobs(x.clamp(min=torch.finfo(torch.float32).min), t, 8)
    check_logprobs(x.clamp(min=torch.finfo(torch.bfloat16).min).to(torch.bfloat16), t, 8)


def test_logprobs_join_of_many_parts():
    """One row in up to 64 parts, few and many alternatives (both forms of the join)."""
    gen = torch.Generator().manual_seed(1)
    for V, k in ((300000, 3), (300000, 32), (70000, 20)):
        x = torch.randn((1, V), generator=gen) * 3
        check_logprobs(x.to(torch.bfloat16), torch.tensor([V // 2]), k)


def test_logprobs_no_rows_and_ignored_targets():
    got = om.token_logprobs(torch.zeros((0, 100), device="cuda"), torch.zeros((0,), dtype=torch.int64, device="cuda"), 3)
    assert [tuple(g.shape) for g in got] == [(0,), (0,), (0,), (0, 3), (0, 3)]
    x = torch.randn((3, 100), device="cuda")
    got = om.token_logprobs(x, torch.tensor([-1, 100, -100], device="cuda"))
    assert bool((got[0] == 0).all())


# ---------------------------------------------------------------- graphs

def test_operators_captured_in_a_graph():
    """One capture of the four operators and the gradient; replays on new inputs, eager calls between them."""
    M, K, N, R, G, E, F, V = 9, 256, 512, 16, 4, 8, 128, 9001
    c = [t.cuda() for t in lora_case(M, K, K, R, G, "bf16", 0, 1)]
    l = [t.cuda() for t in layer_case(M, K, F, E, 2, "bf16", 0, 2)]
    Wv = draw(torch.Generator().manual_seed(3), (K, V), K ** -0.5, "bf16").cuda()
    targets = torch.randint(0, V, (M,), device="cuda")
    gl = torch.randn((M,), device="cuda")
    X = c[0].clone()

    def step(ws):
        Y, w0 = om.lora_matmul(X, *c[1:], workspace=ws[0])
        ids, w = om.moe_route(l[1], 2)
        Z, w1 = om.moe_layer(Y, l[1], 2, *l[2:], workspace=ws[1])
        logits = om.matmul(Z, Wv)
        out = om.token_logprobs(logits, targets, 5)
        g = om.token_logprobs_grad(logits, targets, out[2], gl, out[1], gl)
        return (Y, ids, w, Z) + tuple(out) + (g,), (w0, w1)

    _, ws = step((None, None))
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step(ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs, _ = step(ws)
    torch.cuda.synchronize()
    for i in range(4):
        X.copy_(torch.randn_like(X))
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        captured = [o.clone() for o in outs]
        eager, _ = step((None, None))
        torch.cuda.synchronize()
        for a, b in zip(captured, eager):
            assert torch.equal(a, b)


# ---------------------------------------------------------------- the native binding

def test_binding_refusals_on_gpu_tensors():
    x = torch.randn((4, 16), device="cuda")
    with pytest.raises(ValueError):
        om.moe_route(x.t(), 2)                                  # not contiguous
    with pytest.raises(ValueError):
        om.moe_route(torch.randn(4, 16), 2)                     # on the host
    with pytest.raises(ValueError):
        om.moe_route(x[0], 2)                                   # 1-d
    with pytest.raises(TypeError):
        om.moe_route([1.0], 2)
    with pytest.raises(TypeError):
        om.moe_route(x.to(torch.complex64), 2)
    with pytest.raises(om.OmmError) as e:
        om.moe_route(x, 17)                                     # more than there are
    assert e.value.code == -3 or e.value.code < 0
    with pytest.raises(om.OmmError):
        om.moe_route(x, 2, indices=torch.empty((4, 2), device="cuda"))  # indices of a float type
    with pytest.raises(om.OmmError):
        om.token_logprobs(x, torch.zeros((5,), dtype=torch.int64, device="cuda"))
    with pytest.raises(om.OmmError):
        om.token_logprobs(x, torch.zeros((4,), dtype=torch.int64, device="cuda"), top_k=33)
    W = torch.randn((16, 16), device="cuda")
    A, B = torch.randn((2, 16, 4), device="cuda"), torch.randn((2, 4, 16), device="cuda")
    idx = torch.zeros((4,), dtype=torch.int32, device="cuda")
    with pytest.raises(om.OmmError):
        om.lora_matmul(x, W, A, B, idx, workspace=torch.empty((256,), dtype=torch.uint8, device="cuda")[:16])
    with pytest.raises(om.OmmError):
        om.lora_matmul(x, W.to(torch.bfloat16), A, B, idx)
    om.lora_matmul(x, W, A, B, idx)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("trans", [0, 1])
def test_lora_more_rows_than_streamed(dt, trans):
    """65536 rows and more that the tiles do not take: the adapters' term first, then the dense product."""
    for M, K, N, R, G in ((66001, 33, 41, 9, 5), (65600, 33, 41, 16, 1100)):
        c = lora_case(M, K, N, R, G, dt, trans, M)
        got, _ = run_lora(c, trans)
        sel = torch.cat([torch.arange(0, M, 997), torch.tensor([M - 2, M - 1])])
        want, tol = lora(c[0][sel], c[1], c[2], c[3], c[4][sel], c[5], c[6], trans, dt)
        assert_within(got[sel.cuda()], want, tol)
