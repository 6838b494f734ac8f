"""Refusals of the decode-side operators: every invalid argument is found on
the host, before any launch.  No call here reaches a kernel."""
import ctypes

import pytest

om = pytest.importorskip("onnx_matmul_family_amd._omm")

from tests.test_abi_cpu import BF16, F16, F32, F64, FAKE, I8, I32, I64, T  # noqa: E402

R = ctypes.byref


def opt(t):
    return R(t) if t is not None else None


def lora_args(M=4, K=8, N=6, r=2, G=3, trans=0, dt=BF16):
    return dict(X=T((M, K), dt), W=T((N, K) if trans else (K, N), dt), A=T((G, r, K) if trans else (G, K, r), dt),
                B=T((G, N, r) if trans else (G, r, N), dt), idx=T((M,), I32), scale=T((G,), F32), bias=T((N,), dt),
                trans=trans, Y=T((M, N), dt), ws=FAKE, n=1 << 30)


def lora_call(a):
    return om.lib().omm_lora_matmul(opt(a["X"]), opt(a["W"]), opt(a["A"]), opt(a["B"]), opt(a["idx"]),
                                    opt(a["scale"]), opt(a["bias"]), a["trans"], opt(a["Y"]), a["ws"], a["n"], None)


@pytest.mark.parametrize("trans", [0, 1])
@pytest.mark.parametrize("change,code", [
    (dict(X=None), -1), (dict(Y=None), -1), (dict(X=T((4, 8), BF16, 0)), -1), (dict(W=T((8, 6), F16)), -2),
    (dict(idx=T((4,), F32)), -2), (dict(scale=T((3,), BF16)), -2), (dict(bias=T((6,), F32)), -2),
    (dict(idx=T((5,), I32)), -3), (dict(scale=T((4,), F32)), -3), (dict(bias=T((5,), BF16)), -3),
    (dict(Y=T((4, 7), BF16)), -3), (dict(W=T((9, 9), BF16)), -3), (dict(A=T((3, 9, 9), BF16)), -3),
    (dict(B=T((2, 2, 6), BF16)), -3), (dict(X=T((4, 8, 1), BF16)), -3), (dict(ws=None), -6), (dict(n=255), -6),
    (dict(ws=FAKE + 16), -6)])
def test_lora_refusals(change, code, trans):
    a = lora_args(trans=trans)
    a.update(change)
    assert lora_call(a) == code


def test_lora_limits_and_empty():
    assert lora_call(lora_args(dt=F64)) == -5
    assert lora_call(lora_args(dt=I8)) == -2
    assert lora_call(lora_args(r=257)) == -5
    assert lora_call(lora_args(M=0)) == 0 and lora_call(lora_args(N=0)) == 0
    size = om.lib().omm_lora_matmul_workspace_size
    assert size(4, 8, 6, 2, BF16) > 0 and size(4, 8, 6, 2, I8) == 0 and size(0, 8, 6, 2, BF16) == 0
    assert size(4096, 8, 6, 2, BF16) >= size(4, 8, 6, 2, BF16)


def route_call(x, k, ids, w):
    return om.lib().omm_moe_route(opt(x), k, 1, opt(ids), opt(w), None)


def test_route_refusals():
    x, ids, w = T((4, 16), F32), T((4, 2), I32), T((4, 2), F32)
    assert route_call(None, 2, ids, w) == -1 and route_call(x, 2, None, w) == -1 and route_call(x, 2, ids, None) == -1
    assert route_call(T((4, 16), F64), 2, ids, w) == -5 and route_call(T((4, 16), I32), 2, ids, w) == -2
    assert route_call(x, 2, T((4, 2), F32), w) == -2 and route_call(x, 2, ids, T((4, 2), BF16)) == -2
    assert route_call(x, 3, ids, w) == -3 and route_call(x, -1, ids, w) == -3
    assert route_call(x, 17, T((4, 17), I32), T((4, 17), F32)) == -3
    assert route_call(T((4, 16, 1), F32), 2, ids, w) == -3
    assert route_call(T((4, 600), F32), 2, ids, w) == -5
    assert route_call(T((4, 64), F32), 17, T((4, 17), I64), T((4, 17), F32)) == -5
    assert route_call(T((0, 16), F32), 2, T((0, 2), I32), T((0, 2), F32)) == 0


def layer_args(M=2, K=8, F=6, E=4, trans=0, dt=BF16):
    up, down = ((E, F, K), (E, K, F)) if trans else ((E, K, F), (E, F, K))
    return dict(X=T((M, K), dt), L=T((M, E), F32), k=2, g=T(up, dt), u=T(up, dt), d=T(down, dt), act=0, trans=trans,
                Y=T((M, K), dt), ws=FAKE, n=1 << 30)


def layer_call(a):
    return om.lib().omm_moe_layer(opt(a["X"]), opt(a["L"]), a["k"], 1, opt(a["g"]), opt(a["u"]), opt(a["d"]),
                                  a["act"], a["trans"], opt(a["Y"]), a["ws"], a["n"], None)


@pytest.mark.parametrize("trans", [0, 1])
@pytest.mark.parametrize("change,code", [
    (dict(X=None), -1), (dict(d=None), -1), (dict(u=T((4, 8, 6), F16)), -2), (dict(L=T((2, 4), I32)), -2),
    (dict(L=T((2, 4), F64)), -5), (dict(L=T((3, 4), F32)), -3), (dict(L=T((2, 5), F32)), -3),
    (dict(u=T((4, 7, 6), BF16)), -3), (dict(d=T((4, 5, 5), BF16)), -3), (dict(Y=T((2, 6), BF16)), -3),
    (dict(k=0), -3), (dict(k=5), -3), (dict(act=2), -5), (dict(ws=None), -6), (dict(n=100), -6),
    (dict(ws=FAKE + 64), -6)])
def test_layer_refusals(change, code, trans):
    a = layer_args(trans=trans)
    a.update(change)
    assert layer_call(a) == code


def test_layer_limits_and_empty():
    assert layer_call(layer_args(M=65)) == -5
    assert layer_call(layer_args(E=513)) == -5
    a = layer_args(E=32)
    a["k"] = 17
    assert layer_call(a) == -5
    assert layer_call(layer_args(dt=F64)) == -5 and layer_call(layer_args(dt=I8)) == -2
    assert layer_call(layer_args(M=0)) == 0
    size = om.lib().omm_moe_layer_workspace_size
    assert size(2, 8, 6, 4, 2) > 0 and size(0, 8, 6, 4, 2) == 0


def lp_args(M=3, V=10, k=2, dt=BF16):
    return dict(x=T((M, V), dt), t=T((M,), I64), k=k, lp=T((M,), F32), e=T((M,), F32), l=T((M,), F32),
                ids=T((M, k), I32), tl=T((M, k), F32), ws=FAKE, n=1 << 30)


def lp_call(a):
    return om.lib().omm_token_logprobs(opt(a["x"]), opt(a["t"]), a["k"], opt(a["lp"]), opt(a["e"]), opt(a["l"]),
                                       opt(a["ids"]), opt(a["tl"]), a["ws"], a["n"], None)


@pytest.mark.parametrize("change,code", [
    (dict(x=None), -1), (dict(t=None), -1), (dict(lp=None), -1), (dict(ids=None), -1), (dict(tl=None), -1),
    (dict(x=T((3, 10), F64)), -5), (dict(x=T((3, 10), I8)), -2), (dict(t=T((3,), F32)), -2), (dict(lp=T((3,), BF16)), -2),
    (dict(ids=T((3, 2), I64)), -2), (dict(tl=T((3, 2), BF16)), -2), (dict(t=T((4,), I32)), -3), (dict(e=T((4,), F32)), -3),
    (dict(l=T((3, 1), F32)), -3), (dict(ids=T((3, 3), I32)), -3), (dict(k=-1), -3), (dict(k=11), -3),
    (dict(x=T((3, 0), BF16)), -3), (dict(x=T((30,), BF16)), -3)])
def test_logprobs_refusals(change, code):
    a = lp_args()
    a.update(change)
    assert lp_call(a) == code


def test_logprobs_limits_workspace_and_empty():
    assert lp_call(lp_args(V=64, k=33)) == -5
    assert lp_call(lp_args(M=0)) == 0
    size = om.lib().omm_token_logprobs_workspace_size
    assert size(1, 131072, 5) > 0 and size(2048, 50001, 20) == 0  # one row is split, many are not
    a = lp_args(M=1, V=131072)
    a["n"] = size(1, 131072, 2) - 1
    assert lp_call(a) == -6
    a["n"], a["ws"] = 1 << 30, FAKE + 8
    assert lp_call(a) == -6


def test_logprobs_grad_refusals():
    x, t, v = T((3, 10), BF16), T((3,), I32), T((3,), F32)

    def call(x=x, t=t, lse=v, ent=v, gl=v, gh=v, d=x):
        return om.lib().omm_token_logprobs_grad(opt(x), opt(t), opt(lse), opt(ent), opt(gl), opt(gh), opt(d), None)
    assert call(x=None) == -1 and call(lse=None) == -1 and call(gl=None) == -1 and call(d=None) == -1
    assert call(ent=None) == -1
    assert call(d=T((3, 10), F32)) == -2 and call(t=T((3,), F32)) == -2 and call(lse=T((3,), BF16)) == -2
    assert call(x=T((3, 10), F64), d=T((3, 10), F64)) == -5
    assert call(d=T((3, 9), BF16)) == -3 and call(t=T((4,), I32)) == -3 and call(gh=T((4,), F32)) == -3
    assert call(x=T((0, 10), BF16), t=T((0,), I32), lse=T((0,), F32), ent=None, gl=T((0,), F32), gh=None,
                d=T((0, 10), BF16)) == 0


def test_binding_refusals():
    import torch
    z = torch.zeros
    with pytest.raises(ValueError):
        om.lora_matmul(z(2, 3), z(3), z(1, 3, 2), z(1, 2, 4), z(2, dtype=torch.int32))
    with pytest.raises(ValueError):
        om.moe_layer(z(2, 4), z(2, 3), 1, z(3, 4, 4), z(3, 4, 4), z(3, 4, 4), activation="relu")
    with pytest.raises(ValueError):  # host tensors
        om.token_logprobs(z(2, 4), z(2, dtype=torch.int64))
