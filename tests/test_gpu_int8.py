"""quantize_rows and int8_matmul against their definitions in 64 bits."""
import math

import pytest
import torch

from tests.decode_util import TORCH, assert_within
from tests.train_util import int8_product, quantise

pytestmark = pytest.mark.gpu

om = pytest.importorskip("onnx_matmul_family_amd._omm")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    om.lib()


def rows(M, K, dt, seed=0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((M, K), generator=gen) * (torch.rand((M, 1), generator=gen) * 3 + 0.01)
    return x.to(TORCH[dt])


def check_quantised(X):
    q, s = om.quantize_rows(X.cuda())
    wq, ws = quantise(X)
    assert q.dtype == torch.int8 and s.dtype == torch.float32
    bad = (q.cpu() != wq)
    assert not bad.any(), (int(bad.sum()), X[bad][:4], q.cpu()[bad][:4], wq[bad][:4])
    assert torch.equal(s.cpu().nan_to_num(-1.0), ws.nan_to_num(-1.0))


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("M,K", [(1, 1), (3, 7), (5, 64), (2, 255), (4, 256), (7, 511), (3, 1000), (2, 2048), (3, 2049),
                                 (2, 4095), (1, 8192), (3, 8200), (2, 16391), (1, 32768), (2, 40003), (300, 72),
                                 (1, 0), (0, 5)])
def test_quantize_rows(M, K, dt):
    check_quantised(rows(M, K, dt, seed=M + K))


def test_quantize_every_pair_of_significands():
    """Ties and near ties: every bf16 x against every bf16 largest value of one binade, and their halves."""
    sig = torch.arange(128, 256, dtype=torch.float32)
    x = torch.cat([sig / 2 ** k for k in range(0, 10)])
    X = torch.cat([x[None, :].expand(128, -1).clamp(max=1e9).minimum(sig[:, None]), sig[:, None]], 1)
    check_quantised(X.to(torch.bfloat16))
    check_quantised(-X.to(torch.float16))
    check_quantised(X * 2.0 ** -120)


def test_quantize_borders_of_fp32():
    """Values within a few units in the last place of the border of two steps."""
    gen = torch.Generator().manual_seed(5)
    amax = torch.rand((64, 1), generator=gen) + 0.5
    h = torch.arange(-127, 127, dtype=torch.float64)[None, :] + 0.5
    near = (h * amax.double() / 127).float()
    X = torch.cat([amax] + [(near.view(torch.int32) + d).view(torch.float32) for d in (-2, -1, 0, 1, 2)], 1)
    check_quantised(X)


@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_quantize_special_rows(dt):
    X = rows(9, 300, dt)
    X[1] = 0
    X[2, 17] = math.inf
    X[3, 299] = -math.inf
    X[4, 0] = math.nan
    X[5] = 0
    X[5, 5] = torch.finfo(TORCH[dt]).smallest_normal * torch.finfo(TORCH[dt]).eps  # the smallest of all
    X[6] = -0.0
    X[7, 3] = torch.finfo(TORCH[dt]).max
    check_quantised(X)


def case(M, K, N, dt, bias, seed=0):
    gen = torch.Generator().manual_seed(seed)
    X = rows(M, K, dt, seed)
    W = torch.randint(-128, 128, (N, K), generator=gen, dtype=torch.int64).to(torch.int8)
    sb = torch.rand((N,), generator=gen) * 0.02 + 1e-4
    b = (torch.randn((N,), generator=gen)).to(TORCH[dt]) if bias else None
    return X, W, sb, b


def check_product(M, K, N, dt, bias, seed=0):
    X, W, sb, b = case(M, K, N, dt, bias, seed)
    q, sa = quantise(X)
    want, tol = int8_product(q, sa, W, sb, b, dt)
    bc = b.cuda() if bias else None
    got, ws = om.int8_matmul(X.cuda(), W.cuda(), sb.cuda(), bias=bc)
    assert got.dtype == X.dtype and got.shape == (M, N) and ws is not None
    assert_within(got, want, tol, "quantised by the call")
    other, none = om.int8_matmul(q.cuda(), W.cuda(), sb.cuda(), a_scale=sa.cuda(), bias=bc, dtype=X.dtype)
    assert none is None or K % 16
    assert torch.equal(other, got)


SHAPES = [(1, 16, 1), (1, 64, 16), (1, 4096, 100), (2, 128, 48), (3, 1000, 77), (5, 2048, 130), (16, 512, 256), (17, 96, 33),
          (31, 272, 65), (33, 1024, 300), (43, 4096, 264), (64, 640, 129), (65, 256, 128), (100, 384, 200),
          (128, 128, 128), (129, 144, 257), (200, 2000, 136), (256, 256, 256), (300, 1008, 515), (512, 128, 384),
          (513, 272, 40)]
ODD = [(1, 1, 1), (1, 5, 3), (1, 4097, 19), (2, 15, 17), (4, 33, 5), (16, 127, 64), (43, 257, 100), (70, 2005, 129),
       (130, 65, 131), (257, 1001, 140)]


@pytest.mark.parametrize("M,K,N", SHAPES + ODD)
@pytest.mark.parametrize("dt,bias", [("bf16", False), ("f16", True), ("f32", True)])
def test_product(M, K, N, dt, bias):
    check_product(M, K, N, dt, bias, seed=M + K + N)


@pytest.mark.parametrize("M,K,N", [(2048, 256, 8192), (4096, 384, 4096), (4097, 128, 4100)])
def test_many_tiles(M, K, N):
    check_product(M, K, N, "bf16", True)


@pytest.mark.parametrize("M", [1, 20, 200])
def test_full_range_sums(M):
    """The largest contraction of -128 and 127 fits 32 bits."""
    K, N = 131071, 5
    q = torch.full((M, K), -128, dtype=torch.int8)
    W = torch.full((N, K), -128, dtype=torch.int8)
    W[1] = 127
    one = torch.ones
    got, _ = om.int8_matmul(q.cuda(), W.cuda(), one(N).cuda(), a_scale=one(M).cuda(), dtype=torch.float32)
    want, tol = int8_product(q, one(M), W, one(N), None, "f32")
    assert_within(got, want, tol)


@pytest.mark.parametrize("M,N", [(1, 8), (40, 40), (130, 130)])
def test_non_finite_rows_and_scales(M, N):
    """A row that is not finite is NaN, the others as without it; scales of 0, NaN and infinity act on theirs."""
    X, W, sb, _ = case(M, 96, N, "bf16", False)
    base, _ = om.int8_matmul(X.cuda(), W.cuda(), sb.cuda())
    Y = X.clone()
    Y[M // 2, 3] = math.nan
    sb[N - 1], sb[N // 2], sb[0] = 0.0, math.nan, math.inf
    got, _ = om.int8_matmul(Y.cuda(), W.cuda(), sb.cuda())
    got, base = got.cpu(), base.cpu()
    keep = torch.ones(N, dtype=torch.bool)
    keep[[0, N // 2, N - 1]] = False
    rest = torch.arange(M) != M // 2
    assert got[M // 2].isnan().all()
    assert torch.equal(got[rest][:, keep], base[rest][:, keep])
    if M > 1:
        assert got[rest][:, N // 2].isnan().all() and (got[rest][:, N - 1] == 0).all()


@pytest.mark.parametrize("M,K,N", [(0, 8, 4), (4, 8, 0), (3, 0, 5)])
@pytest.mark.parametrize("bias", [False, True])
def test_empty(M, K, N, bias):
    check_product(M, K, N, "f16", bias) if M and N else om.int8_matmul(*[t.cuda() for t in case(M, K, N, "f16", False)[:3]])


@pytest.mark.parametrize("off", [1, 4, 8, 15])
@pytest.mark.parametrize("M,N", [(1, 50), (16, 64), (90, 140)])
def test_unaligned_bases(M, N, off):
    K = 128
    X, W, sb, _ = case(M, K, N, "bf16", False)
    q, sa = quantise(X)
    pool = torch.zeros((N * K + 64,), dtype=torch.int8, device="cuda")
    pool[off:off + N * K] = W.cuda().reshape(-1)
    qpool = torch.zeros((M * K + 64,), dtype=torch.int8, device="cuda")
    qpool[off:off + M * K] = q.cuda().reshape(-1)
    y = torch.full((M * N + 64,), 7.0, device="cuda", dtype=torch.bfloat16)
    out = y[off:off + M * N].view(M, N)
    om.int8_matmul(qpool[off:off + M * K].view(M, K), pool[off:off + N * K].view(N, K), sb.cuda(), a_scale=sa.cuda(), Y=out)
    want, tol = int8_product(q, sa, W, sb, None, "bf16")
    assert_within(out, want, tol)
    assert (y[:off] == 7).all() and (y[off + M * N:] == 7).all()


@pytest.mark.parametrize("M,K,N", [(1, 64, 33), (43, 100, 70), (130, 128, 129), (256, 128, 256)])
def test_nothing_outside_the_outputs(M, K, N):
    X, W, sb, _ = case(M, K, N, "f32", False)
    guard = 256
    y = torch.full((M * N + 2 * guard,), 7.0, device="cuda")
    om.int8_matmul(X.cuda(), W.cuda(), sb.cuda(), Y=y[guard:guard + M * N].view(M, N))
    assert (y[:guard] == 7).all() and (y[guard + M * N:] == 7).all()
    q = torch.full((M * K + 2 * guard,), 7, device="cuda", dtype=torch.int8)
    s = torch.full((M + 2 * guard,), 7.0, device="cuda")
    om.quantize_rows(X.cuda(), q[guard:guard + M * K].view(M, K), s[guard:guard + M])
    for t, n in ((q, M * K), (s, M)):
        assert (t[:guard] == 7).all() and (t[guard + n:] == 7).all()


@pytest.mark.parametrize("adt,ydt", [("f32", "bf16"), ("bf16", "f32"), ("f16", "bf16")])
@pytest.mark.parametrize("M", [3, 100])
def test_types_of_input_and_output_differ(adt, ydt, M):
    X, W, sb, _ = case(M, 160, 72, adt, False)
    q, sa = quantise(X)
    got, _ = om.int8_matmul(X.cuda(), W.cuda(), sb.cuda(), dtype=TORCH[ydt])
    want, tol = int8_product(q, sa, W, sb, None, ydt)
    assert got.dtype == TORCH[ydt]
    assert_within(got, want, tol)


def test_weights_by_rows_in_a_run():
    """As a program uses them: weights quantised once, several projections of one input."""
    gen = torch.Generator().manual_seed(3)
    X = torch.randn((37, 320), generator=gen).to(torch.bfloat16)
    Ws = [torch.randn((n, 320), generator=gen).to(torch.bfloat16) for n in (320, 80, 80)]
    packed = [om.quantize_rows(W.cuda()) for W in Ws]
    q, s = om.quantize_rows(X.cuda())
    for W, (wq, sw) in zip(Ws, packed):
        y, _ = om.int8_matmul(q, wq, sw, a_scale=s)
        want, tol = int8_product(*quantise(X), *quantise(W), None, "bf16")
        assert_within(y, want, tol + 4 * 2.0 ** -24 * want.abs())
        # near the product of what was quantised: every value is off by at most half a step of its row
        full = X.double() @ W.double().t()
        sx, sv = X.double().abs().amax(1) / 127, W.double().abs().amax(1) / 127
        bound = 0.5 * (sx[:, None] * W.double().abs().sum(1)[None, :] + X.double().abs().sum(1)[:, None] * sv[None, :]) \
            + 0.25 * 320 * sx[:, None] * sv[None, :]
        assert ((y.double().cpu() - full).abs() <= bound + 2.0 ** -8 * full.abs() + 1e-3).all()


@pytest.mark.parametrize("M,K,N", [(200, 257, 2080), (1100, 65, 500), (300, 2005, 2048), (130, 33, 4100)])
@pytest.mark.parametrize("dt,bias", [("bf16", False), ("f16", True), ("f32", True)])
def test_odd_rows_copied(M, K, N, dt, bias):
    check_product(M, K, N, dt, bias, seed=M + K)


@pytest.mark.parametrize("off", [1, 6])
@pytest.mark.parametrize("M,K,N", [(1100, 65, 500), (700, 99, 512), (3, 131, 40), (64, 127, 8200)])
def test_odd_rows_at_any_base(M, K, N, off):
    """Streamed and copied rows of odd lengths that start anywhere, between other data."""
    gen = torch.Generator().manual_seed(M + off)
    buf_a = torch.randint(-128, 128, (M * K + off + 8,), generator=gen).to(torch.int8).cuda()
    buf_b = torch.randint(-128, 128, (N * K + off + 9,), generator=gen).to(torch.int8).cuda()
    a, b = buf_a[off:off + M * K].view(M, K), buf_b[off + 1:off + 1 + N * K].view(N, K)
    sa, sb = torch.rand((M,), generator=gen).cuda(), torch.rand((N,), generator=gen).cuda()
    got, _ = om.int8_matmul(a, b, sb, a_scale=sa, dtype=torch.float32)
    want, tol = int8_product(a.cpu(), sa.cpu(), b.cpu(), sb.cpu(), None, "f32")
    assert_within(got, want, tol, "product")
