"""moe_route and moe_layer on the GPU against the 64-bit forms of
tests/decode_util.py (which derives the bounds)."""
import math

import pytest
import torch

from tests.decode_util import TORCH, assert_within, draw, moe, route, route_tol

pytestmark = pytest.mark.gpu

om = pytest.importorskip("onnx_matmul_family_amd._omm")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    om.lib()


def check_route(x, k, renorm, what=""):
    ids, w = route(x, k, renorm)
    gi, gw = om.moe_route(x.cuda(), k, renormalize=renorm)
    torch.cuda.synchronize()
    assert torch.equal(gi.cpu().to(torch.int64), ids), what
    assert_within(gw, w, route_tol(x, ids, w).nan_to_num(nan=0.0), what)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,E,k", [(1, 1, 1), (3, 4, 4), (5, 8, 2), (2, 60, 6), (7, 64, 8), (130, 65, 3), (4, 128, 16),
                                   (3, 160, 6), (2, 256, 8), (5, 511, 16), (2, 512, 1)])
@pytest.mark.parametrize("renorm", [True, False])
def test_route(M, E, k, dt, renorm):
    gen = torch.Generator().manual_seed(M + 7 * E + k)
    check_route(draw(gen, (M, E), 2.0, dt), k, renorm)


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("E", [5, 64, 200])
def test_route_ties_and_masks(E, renorm):
    x = torch.zeros((8, E))
    x[1] = -math.inf                      # nothing left
    x[2, 1:] = -math.inf                  # fewer than k left
    x[3, E // 2] = math.nan
    x[4] = torch.arange(E) % 3            # ties in bands
    x[5] = -torch.arange(E) * 40.0        # far apart: small weights vanish
    x[6] = torch.finfo(torch.float32).min
    x[6, E - 1] = 0.0
    x[7] = torch.arange(E) % 2 * -0.0     # zeros of both signs tie
    check_route(x, 4, renorm)


def test_route_int64_output_and_stream():
    gen = torch.Generator().manual_seed(1)
    x = draw(gen, (9, 64), 2.0, "f32")
    out = torch.full((11, 8), -7, dtype=torch.int64, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    om.moe_route(x.cuda(), 8, indices=out[1:10], stream=s)
    s.synchronize()
    assert torch.equal(out[1:10].cpu(), route(x, 8, True)[0])
    assert bool((out[0] == -7).all()) and bool((out[10] == -7).all())


def layer_case(M, K, F, E, k, dt, trans, seed):
    gen = torch.Generator().manual_seed(seed)
    X = draw(gen, (M, K), 1.0, dt)
    logits = torch.randn((M, E), generator=gen) * 2
    up, down = ((E, F, K), (E, K, F)) if trans else ((E, K, F), (E, F, K))
    return (X, logits, draw(gen, up, K ** -0.5, dt), draw(gen, up, K ** -0.5, dt), draw(gen, down, F ** -0.5, dt))


def check_layer(X, logits, k, Wg, Wu, Wd, dt, trans, renorm=True, activation="silu", Y=None):
    want, tol = moe(X, logits, k, Wg, Wu, Wd, renorm, activation, trans, dt)
    got, _ = om.moe_layer(X.cuda(), logits.cuda(), k, Wg.cuda(), Wu.cuda(), Wd.cuda(), renormalize=renorm,
                          activation=activation, trans=trans, Y=Y)
    torch.cuda.synchronize()
    assert_within(got, want, tol)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("trans", [0, 1])
@pytest.mark.parametrize("M,K,F,E,k", [(1, 64, 64, 4, 2), (1, 512, 256, 8, 3), (3, 136, 72, 5, 5), (16, 256, 128, 4, 1),
                                       (17, 128, 200, 6, 2), (33, 96, 160, 3, 3), (64, 64, 64, 9, 4),
                                       (1, 8, 8, 1, 1), (2, 7, 5, 3, 2), (5, 130, 66, 4, 2), (20, 63, 33, 2, 2),
                                       (1, 1, 1, 1, 1), (4, 1032, 520, 70, 6)])
def test_layer(M, K, F, E, k, dt, trans):
    case = layer_case(M, K, F, E, k, dt, trans, M + K + F)
    check_layer(case[0], case[1], k, *case[2:], dt, trans, renorm=bool(M % 2), activation="gelu" if K % 3 else "silu")


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("trans", [0, 1])
def test_layer_all_tokens_one_expert_and_masked_tokens(dt, trans):
    """64 tokens on one expert; a token with one expert left; a token with none (output 0)."""
    M, K, F, E, k = 64, 256, 192, 8, 2
    X, logits, Wg, Wu, Wd = layer_case(M, K, F, E, k, dt, trans, 5)
    logits[:, 3] += 100
    logits[7] = -math.inf
    logits[9] = -math.inf
    logits[9, 6] = 0.0
    check_layer(X, logits, k, Wg, Wu, Wd, dt, trans)
    Y, _ = om.moe_layer(X.cuda(), logits.cuda(), k, Wg.cuda(), Wu.cuda(), Wd.cuda(), trans=trans)
    assert bool((Y[7] == 0).all())


def test_layer_large_fp16_intermediate():
    """Branch products far beyond fp16's range (the layer holds them in fp32)."""
    M, K, F, E, k = 3, 64, 64, 2, 1
    X, logits, Wg, Wu, Wd = layer_case(M, K, F, E, k, "f16", 0, 6)
    X, Wg, Wu = X * 64, Wg * 32, Wu * 32
    Wd = Wd * 2.0 ** -10
    check_layer(X, logits, k, Wg, Wu, Wd, "f16", 0)


@pytest.mark.parametrize("off", [1, 4])
def test_layer_unaligned_weights_and_canaries(off):
    M, K, F, E, k = 3, 64, 72, 4, 2
    X, logits, Wg, Wu, Wd = layer_case(M, K, F, E, k, "bf16", 0, 8)
    logits = logits.to(torch.bfloat16)
    want, tol = moe(X, logits, k, Wg, Wu, Wd, True, "silu", 0, "bf16")
    bufs = []
    for w in (Wg, Wu, Wd):
        b = torch.zeros(w.numel() + off, dtype=torch.bfloat16, device="cuda")
        b[off:].view(w.shape).copy_(w)
        bufs.append(b[off:].view(w.shape))
    out = torch.full((M + 2, K), 9.0, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    om.moe_layer(X.cuda(), logits.cuda(), k, *bufs, Y=out[1:-1], stream=s)
    s.synchronize()
    assert_within(out[1:-1], want, tol)
    assert bool((out[0] == 9).all()) and bool((out[-1] == 9).all())


@pytest.mark.parametrize("M", [1, 9, 40])
def test_layer_repeats_bit_for_bit(M):
    """No result depends on the order in which workgroups finish; a used workspace changes nothing."""
    X, logits, Wg, Wu, Wd = [t.cuda() for t in layer_case(M, 512, 384, 16, 4, "bf16", 0, M)]
    Y, ws = om.moe_layer(X, logits, 4, Wg, Wu, Wd)
    first = Y.clone()
    ws.fill_(255)
    for _ in range(5):
        Y2, _ = om.moe_layer(X, logits, 4, Wg, Wu, Wd, workspace=ws)
        assert torch.equal(Y2.view(torch.int16), first.view(torch.int16))


def test_layer_past_32_bit_offsets():
    M, K, F, E, k = 2, 8192, 4096, 70, 1  # 2.3e9 elements of each weight
    gen = torch.Generator().manual_seed(2)
    X = draw(gen, (M, K), 1.0, "bf16")
    Wg, Wu = (torch.zeros((E, K, F), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    Wd = torch.zeros((E, F, K), dtype=torch.bfloat16, device="cuda")
    g, u, d = draw(gen, (1, K, F), K ** -0.5, "bf16"), draw(gen, (1, K, F), K ** -0.5, "bf16"), \
        draw(gen, (1, F, K), F ** -0.5, "bf16")
    Wg[-1], Wu[-1], Wd[-1] = g[0].cuda(), u[0].cuda(), d[0].cuda()
    logits = torch.zeros((M, E))
    logits[:, -1] = 5.0
    want, tol = moe(X, torch.zeros((M, 1)), 1, g, u, d, True, "silu", 0, "bf16")
    got, _ = om.moe_layer(X.cuda(), logits.cuda(), k, Wg, Wu, Wd)
    assert_within(got, want, tol)
