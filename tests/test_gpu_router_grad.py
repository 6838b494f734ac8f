"""moe_balance and moe_route_grad against their definitions in 64 bits and against differences."""
import math

import pytest
import torch

from tests.decode_util import TORCH, assert_within
from tests.train_util import balance, route_grad

pytestmark = pytest.mark.gpu

om = pytest.importorskip("onnx_matmul_family_amd._omm")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    om.lib()


def case(M, E, k, dt, padded=0.0, seed=0):
    gen = torch.Generator().manual_seed(seed)
    x = (torch.randn((M, E), generator=gen) * 1.5 + torch.randn((1, E), generator=gen) * 0.5).to(TORCH[dt])
    ids = torch.topk(x.float(), k, dim=1)[1].to(torch.int32)
    mask = (torch.rand((M,), generator=gen) >= padded) if padded else None
    g = torch.randn((M, k), generator=gen)
    return x, ids, mask, g


def gpu(t):
    return t.cuda() if t is not None else None


def check_balance(x, ids, mask):
    losses, counts, tokens = om.moe_balance(x.cuda(), ids.cuda(), token_mask=gpu(mask))
    (wl, wc, n), tol = balance(x, ids, mask)
    assert losses.dtype == torch.float32 and counts.dtype == tokens.dtype == torch.int32
    assert torch.equal(counts.cpu().long(), wc) and int(tokens) == n
    assert_within(losses, wl, tol + 1e-37, "losses")
    return losses, counts, tokens


def check_grad(x, ids, mask, g, renorm, dt, gl, counts=None, tokens=None, **kw):
    got = om.moe_route_grad(x.cuda(), ids.cuda(), gpu(g), renormalize=renorm, token_mask=gpu(mask), counts=counts,
                            tokens=tokens, grad_losses=gpu(gl), **kw)
    c = counts.cpu().long() if counts is not None else None
    want, tol = route_grad(x, ids, g, renorm, mask, c, int(tokens) if tokens is not None else 0, gl, dt)
    assert got.dtype == x.dtype
    assert_within(got, want, tol, "gradient")
    return got


SIZES = [(1, 1, 1), (1, 8, 2), (3, 5, 5), (16, 16, 4), (17, 17, 1), (100, 60, 4), (333, 64, 8), (1000, 65, 8), (50, 128, 16),
         (70, 160, 6), (129, 256, 8), (40, 257, 3), (65, 511, 16), (33, 512, 8), (5000, 64, 8), (2000, 512, 2)]


@pytest.mark.parametrize("M,E,k", SIZES)
@pytest.mark.parametrize("dt,padded", [("bf16", 0.0), ("f16", 0.3), ("f32", 0.3)])
def test_losses_and_gradient(M, E, k, dt, padded):
    x, ids, mask, g = case(M, E, k, dt, padded, seed=M + E)
    _, counts, tokens = check_balance(x, ids, mask)
    gl = torch.tensor([0.3 * max(M, 1), 0.1 * max(M, 1)])
    for renorm in (False, True):
        check_grad(x, ids, mask, g, renorm, dt, gl, counts, tokens)


@pytest.mark.parametrize("which", ["weights", "losses", "first", "none"])
def test_parts_of_the_gradient(which):
    x, ids, mask, g = case(90, 24, 3, "f32", 0.2)
    _, counts, tokens = om.moe_balance(x.cuda(), ids.cuda(), token_mask=mask.cuda())
    gl = torch.tensor([50.0, 0.0 if which == "first" else 9.0])
    if which == "weights":
        check_grad(x, ids, mask, g, True, "f32", None)
    elif which == "none":
        assert (check_grad(x, ids, mask, None, True, "f32", None) == 0).all()
    else:
        check_grad(x, ids, mask, None, True, "f32", gl, counts, tokens)


@pytest.mark.parametrize("renorm", [False, True])
def test_against_differences(renorm):
    """Directional differences of the loss as the forward operators compute it."""
    M, E, k = 64, 12, 3
    x, ids, mask, g = case(M, E, k, "f32", 0.2, seed=4)
    gl = torch.tensor([3.0, 2.0])
    _, counts, tokens = om.moe_balance(x.cuda(), ids.cuda(), token_mask=mask.cuda())
    d = om.moe_route_grad(x.cuda(), ids.cuda(), g.cuda(), renormalize=renorm, token_mask=mask.cuda(), counts=counts,
                          tokens=tokens, grad_losses=gl.cuda()).double().cpu()

    def loss(y):
        y = y.double()
        p = torch.softmax(y, 1)
        w = p.gather(1, ids.long())
        if renorm:
            w = w / w.sum(1, keepdim=True)
        f = counts.cpu().double() / counts.sum().item()
        lse = torch.logsumexp(y, 1)
        return ((w * g.double())[mask].sum() + 3.0 * E * (f * p[mask].mean(0)).sum() + 2.0 * (lse[mask] ** 2).mean())

    gen = torch.Generator().manual_seed(9)
    for _ in range(5):
        v = torch.randn((M, E), generator=gen).double()
        h = 1e-5
        diff = float(loss(x.double() + h * v) - loss(x.double() - h * v)) / (2 * h)
        # third derivatives h^2, and fp32 results
        assert abs(diff - float((d * v).sum())) <= 1e-4 * (1 + abs(diff))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_special_rows(dt):
    """Excluded experts, rows with none left, NaN and infinity, padding that holds NaN, indices out of range."""
    x, ids, _, g = case(12, 20, 4, dt)
    x[1, 5:] = -math.inf
    x[2, :] = -math.inf
    x[7, 0] = -math.inf
    mask = torch.ones((12,), dtype=torch.uint8)
    mask[3], mask[4] = 0, 0
    x[3, 2] = math.nan
    x[4, 2] = math.inf
    mask[6] = 255
    ids[5, 1], ids[6, 0], ids[8, 3] = -1, 20, 2 ** 31 - 1
    ids[9, :] = 7  # the same expert four times
    ids[10, :2] = 3
    _, counts, tokens = check_balance(x, ids, mask)
    gl = torch.tensor([5.0, 2.0])
    for renorm in (False, True):
        got = check_grad(x, ids, mask, g, renorm, dt, gl, counts, tokens)
        assert (got[2:5] == 0).all() and torch.isfinite(got.float()).all()
        assert (got[1, 5:] == 0).all()
    # a token that counts and is not finite: its own gradient and the losses are NaN, nothing else
    x[0, 1] = math.nan
    x[11, 1] = math.inf
    losses, c2, t2 = om.moe_balance(x.cuda(), ids.cuda(), token_mask=mask.cuda())
    assert losses.isnan().all() and torch.equal(c2, counts) and torch.equal(t2, tokens)
    got = check_grad(x, ids, mask, g, True, dt, gl, counts, tokens)
    assert got[0].isnan().all() and got[11].isnan().all() and torch.isfinite(got[1:11].float()).all()


def test_no_tokens_and_no_selections():
    x, ids, _, g = case(20, 9, 2, "f32")
    mask = torch.zeros((20,), dtype=torch.bool)
    losses, counts, tokens = check_balance(x, ids, mask)
    assert (losses == 0).all() and (counts == 0).all()
    gl = torch.tensor([1.0, 1.0])
    assert (check_grad(x, ids, mask, g, True, "f32", gl, counts, tokens) == 0).all()
    check_grad(x, ids, None, g, True, "f32", gl, counts, tokens)  # (counts of other tokens: none)
    none = ids[:, :0].contiguous()
    _, counts, tokens = check_balance(x, none, None)
    check_grad(x, none, None, g[:, :0].contiguous(), True, "f32", gl, counts, tokens)
    empty = x[:0].contiguous()
    losses, counts, tokens = check_balance(empty, ids[:0].contiguous(), None)
    assert om.moe_route_grad(empty.cuda(), ids[:0].contiguous().cuda()).shape == (0, 9)


def test_far_logits():
    """lse of far logits, probabilities that underflow."""
    x, ids, _, g = case(30, 33, 4, "f32")
    x[:10] += 1e4
    x[10:20] -= 1e4
    x[20:] *= 300
    ids = torch.topk(x, 4, dim=1)[1].to(torch.int32)
    _, counts, tokens = check_balance(x, ids, None)
    for renorm in (False, True):
        check_grad(x, ids, None, g, renorm, "f32", torch.tensor([1.0, 0.01]), counts, tokens)


def test_index_types_and_in_place():
    x, ids, mask, g = case(77, 30, 5, "bf16", 0.3)
    a = om.moe_balance(x.cuda(), ids.cuda(), token_mask=mask.cuda())
    b = om.moe_balance(x.cuda(), ids.long().cuda(), token_mask=mask.to(torch.uint8).cuda())
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    gl = torch.tensor([4.0, 1.0])
    want = check_grad(x, ids, mask, g, True, "bf16", gl, a[1], a[2])
    y = x.cuda()
    out = om.moe_route_grad(y, ids.long().cuda(), g.cuda(), token_mask=mask.cuda(), counts=a[1], tokens=a[2],
                            grad_losses=gl.cuda(), grad_logits=y)
    assert out.data_ptr() == y.data_ptr() and torch.equal(out, want)


def test_with_the_router():
    """moe_route's selections through the losses and back."""
    gen = torch.Generator().manual_seed(2)
    x = torch.randn((500, 64), generator=gen).to(torch.bfloat16)
    ids, w = om.moe_route(x.cuda(), 6)
    losses, counts, tokens = check_balance(x, ids.cpu(), None)
    assert int(counts.sum()) == 3000 and float(losses[0]) > 1.0
    g = torch.randn((500, 6), generator=gen)
    check_grad(x, ids.cpu(), None, g, True, "bf16", torch.tensor([10.0, 1.0]), counts, tokens)


@pytest.mark.parametrize("M,E", [(40000, 64), (9000, 300)])
def test_same_bits(M, E):
    x, ids, mask, _ = case(M, E, 4, "f32", 0.1)
    x, ids, mask = x.cuda(), ids.cuda(), mask.cuda()
    first = om.moe_balance(x, ids, token_mask=mask)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, om.moe_balance(x, ids, token_mask=mask)))


def test_nothing_outside_the_gradient():
    x, ids, _, g = case(37, 21, 2, "f32")
    y = torch.full((37 * 21 + 512,), 7.0, device="cuda")
    om.moe_route_grad(x.cuda(), ids.cuda(), g.cuda(), grad_logits=y[256:256 + 37 * 21].view(37, 21))
    assert (y[:256] == 7).all() and (y[256 + 37 * 21:] == 7).all()


@pytest.mark.parametrize("M,E,k,dt", [(45000, 72, 4, "bf16"), (30000, 200, 8, "f32"), (23000, 384, 6, "f16"), (21000, 333, 16, "bf16")])
def test_several_turns(M, E, k, dt):
    x, ids, mask, g = case(M, E, k, dt, 0.1, seed=E)
    _, counts, tokens = check_balance(x, ids, mask)
    check_grad(x, ids, mask, g, True, dt, torch.tensor([0.3 * M, 0.1 * M]), counts, tokens)


@pytest.mark.parametrize("E", [40, 72, 160, 320, 512])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("shift", [0, 1])
def test_wide_special_rows(E, dt, shift):
    """The same expert in many selections, none, rows with hardly any expert left, rows that start on any element."""
    x, ids, _, g = case(40, E, 16, dt, seed=E)
    x[1, 1:] = -math.inf
    x[2, : E - 1] = -math.inf
    x[3, :] = -math.inf
    ids[4, :] = E - 1
    ids[5, ::2] = 3
    ids[6, 1::2] = ids[6, 0]
    ids[7, :], ids[8, 3:], ids[9, 5] = -1, E, -2 ** 31
    mask = torch.ones((40,), dtype=torch.bool)
    mask[11] = mask[38] = False
    x[11, 0] = math.nan
    buf = torch.zeros((40 * E + shift,), dtype=x.dtype)
    buf[shift:] = x.reshape(-1)
    y = buf.cuda()[shift:].view(40, E)
    losses, counts, tokens = om.moe_balance(y, ids.cuda(), token_mask=mask.cuda())
    (wl, wc, n), tol = balance(x, ids, mask)
    assert torch.equal(counts.cpu().long(), wc) and int(tokens) == n
    assert_within(losses, wl, tol + 1e-37, "losses")
    gl = torch.tensor([12.0, 3.0])
    for renorm in (False, True):
        want, t = route_grad(x, ids, g, renorm, mask, counts.cpu().long(), n, gl, dt)
        for inplace in (False, True):
            z = y.clone() if not shift else torch.cat([y.new_zeros(shift), y.reshape(-1)])[shift:].view(40, E)
            got = om.moe_route_grad(z, ids.cuda(), g.cuda(), renormalize=renorm, token_mask=mask.cuda(), counts=counts,
                                    tokens=tokens, grad_losses=gl.cuda(), grad_logits=z if inplace else None)
            assert_within(got, want, t, "gradient")
            assert (got[11] == 0).all() and (got[38] == 0).all()
