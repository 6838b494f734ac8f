"""Refusals of the operators that train, balance and quantise: every invalid argument
is found on the host, before any launch.  No call here reaches a kernel."""
import ctypes

import pytest

om = pytest.importorskip("onnx_matmul_family_amd._omm")

from tests.test_abi_cpu import BF16, F16, F32, F64, FAKE, I8, I32, I64, T, U8  # noqa: E402

R = ctypes.byref


def opt(t):
    return R(t) if t is not None else None


def quantise(x, q, s):
    return om.lib().omm_quantize_rows(opt(x), opt(q), opt(s), None)


def test_quantize_refusals():
    x, q, s = T((4, 8), BF16), T((4, 8), I8), T((4,), F32)
    assert quantise(None, q, s) == -1 and quantise(x, None, s) == -1 and quantise(x, q, None) == -1
    assert quantise(T((4, 8), BF16, 0), q, s) == -1
    assert quantise(T((4, 8), F64), q, s) == -5 and quantise(T((4, 8), I8), q, s) == -2
    assert quantise(x, T((4, 8), U8), s) == -2 and quantise(x, q, T((4,), BF16)) == -2
    assert quantise(T((4, 8, 1), BF16), q, s) == -3 and quantise(x, T((4, 9), I8), s) == -3
    assert quantise(x, q, T((8,), F32)) == -3 and quantise(x, q, T((4, 1), F32)) == -3
    assert quantise(T((1, 2 ** 31), BF16), T((1, 2 ** 31), I8), T((1,), F32)) == -5
    assert quantise(T((0, 8), BF16), T((0, 8), I8), T((0,), F32)) == 0


def product(**change):
    a = dict(a=T((4, 32), I8), sa=T((4,), F32), b=T((6, 32), I8), sb=T((6,), F32), bias=T((6,), BF16), Y=T((4, 6), BF16),
             ws=None, n=0)
    a.update(change)
    return om.lib().omm_int8_matmul(opt(a["a"]), opt(a["sa"]), opt(a["b"]), opt(a["sb"]), opt(a["bias"]), opt(a["Y"]),
                                    a["ws"], a["n"], None)


@pytest.mark.parametrize("change,code", [
    (dict(a=None), -1), (dict(b=None), -1), (dict(sb=None), -1), (dict(Y=None), -1), (dict(sa=None), -1),
    (dict(a=T((4, 32), I8, 0)), -1), (dict(a=T((4, 32), U8)), -2), (dict(a=T((4, 32), F64), sa=None), -5),
    (dict(b=T((6, 32), U8)), -2), (dict(sb=T((6,), BF16)), -2), (dict(sa=T((4,), F16)), -2), (dict(Y=T((4, 6), I8)), -2),
    (dict(Y=T((4, 6), F64)), -5), (dict(bias=T((6,), F32)), -2), (dict(a=T((4, 31), I8)), -3),
    (dict(a=T((1, 4, 32), I8)), -3), (dict(b=T((32, 6), I8)), -3), (dict(sa=T((5,), F32)), -3), (dict(sa=T((1,), F32)), -3),
    (dict(sb=T((5,), F32)), -3), (dict(sb=T((1,), F32)), -3), (dict(bias=T((1,), BF16)), -3), (dict(Y=T((6, 4), BF16)), -3),
    (dict(a=T((4, 32), BF16), ws=FAKE, n=1 << 20), -3),  # a scale for rows that have none yet
    (dict(a=T((4, 32), BF16), sa=None), -6), (dict(a=T((4, 32), BF16), sa=None, ws=FAKE, n=100), -6),
    (dict(a=T((4, 32), BF16), sa=None, ws=FAKE + 16, n=1 << 20), -6),
    (dict(a=T((4, 131072), I8), b=T((6, 131072), I8)), -5),
    (dict(a=T((2 ** 28, 32), I8), sa=T((2 ** 28,), F32), b=T((2 ** 28, 32), I8), sb=T((2 ** 28,), F32), bias=None,
          Y=T((2 ** 28, 2 ** 28), BF16)), -5)])
def test_product_refusals(change, code):
    assert product(**change) == code


def test_product_empty_and_size():
    assert product(a=T((0, 32), I8), sa=T((0,), F32), Y=T((0, 6), BF16)) == 0
    assert product(b=T((0, 32), I8), sb=T((0,), F32), bias=None, Y=T((4, 0), BF16)) == 0
    size = om.lib().omm_int8_matmul_workspace_size
    assert size(4, 32, 6, I8) == 0 and size(0, 32, 6, BF16) == 0 and size(4, 131072, 6, BF16) == 0
    assert size(4, 32, 6, F64) == 0 and size(4, -1, 6, BF16) == 0
    assert size(4, 33, 6, BF16) >= 4 * 4 + 4 * 33 and size(4, 33, 6, F32) == size(4, 33, 6, BF16)


def load(**change):
    a = dict(x=T((5, 8), BF16), ids=T((5, 2), I32), mask=T((5,), U8), losses=T((2,), F32), counts=T((8,), I32),
             tokens=T((1,), I32), ws=FAKE, n=1 << 20)
    a.update(change)
    return om.lib().omm_moe_balance(opt(a["x"]), opt(a["ids"]), opt(a["mask"]), opt(a["losses"]), opt(a["counts"]),
                                    opt(a["tokens"]), a["ws"], a["n"], None)


@pytest.mark.parametrize("change,code", [
    (dict(x=None), -1), (dict(ids=None), -1), (dict(losses=None), -1), (dict(counts=None), -1), (dict(tokens=None), -1),
    (dict(mask=T((5,), U8, 0)), -1), (dict(x=T((5, 8), F64)), -5), (dict(x=T((5, 8), I32)), -2), (dict(ids=T((5, 2), F32)), -2),
    (dict(mask=T((5,), I32)), -2), (dict(losses=T((2,), BF16)), -2), (dict(counts=T((8,), I64)), -2),
    (dict(tokens=T((1,), I64)), -2), (dict(x=T((5, 8, 1), BF16)), -3), (dict(ids=T((4, 2), I32)), -3),
    (dict(ids=T((10,), I32)), -3), (dict(mask=T((4,), U8)), -3), (dict(losses=T((3,), F32)), -3),
    (dict(counts=T((9,), I32)), -3), (dict(tokens=T((2,), I32)), -3), (dict(x=T((5, 0), BF16), counts=T((0,), I32)), -3),
    (dict(x=T((5, 513), BF16), counts=T((513,), I32)), -5), (dict(ids=T((5, 17), I32)), -5),
    (dict(x=T((2 ** 27, 8), BF16), ids=T((2 ** 27, 2), I32), mask=None), -5)] + [
    (dict(x=T((300, 8), BF16), ids=T((300, 2), I32), mask=None, **ws), -6)
    for ws in (dict(ws=None), dict(n=64), dict(ws=FAKE + 64))])
def test_balance_refusals(change, code):
    assert load(**change) == code


def grad(**change):
    a = dict(x=T((5, 8), BF16), ids=T((5, 2), I64), g=T((5, 2), F32), mask=T((5,), U8), counts=T((8,), I32),
             tokens=T((1,), I32), gl=T((2,), F32), out=T((5, 8), BF16))
    a.update(change)
    return om.lib().omm_moe_route_grad(opt(a["x"]), opt(a["ids"]), opt(a["g"]), 1, opt(a["mask"]), opt(a["counts"]),
                                       opt(a["tokens"]), opt(a["gl"]), opt(a["out"]), None)


@pytest.mark.parametrize("change,code", [
    (dict(x=None), -1), (dict(ids=None), -1), (dict(out=None), -1), (dict(counts=None), -1), (dict(tokens=None), -1),
    (dict(g=T((5, 2), F32, 0)), -1), (dict(x=T((5, 8), F64), out=T((5, 8), F64)), -5), (dict(out=T((5, 8), F32)), -2),
    (dict(g=T((5, 2), BF16)), -2), (dict(gl=T((2,), F64)), -2), (dict(g=T((5, 3), F32)), -3), (dict(out=T((5, 9), BF16)), -3),
    (dict(gl=T((1,), F32)), -3), (dict(counts=T((7,), I32)), -3), (dict(mask=T((6,), U8)), -3)])
def test_gradient_refusals(change, code):
    assert grad(**change) == code


def test_router_empty():
    assert grad(x=T((0, 8), BF16), ids=T((0, 2), I64), g=None, mask=None, out=T((0, 8), BF16)) == 0
    size = om.lib().omm_moe_balance_workspace_size
    assert size(0, 8) == 0 and size(5, 0) == 0 and size(300, 513) == 0 and size(300, 8) > 0


def ortho(G=T((6, 4), BF16), steps=5, out=T((6, 4), BF16), ws=FAKE, n=1 << 30):
    return om.lib().omm_orthogonalize(opt(G), steps, opt(out), ws, n, None)


def test_orthogonalize_refusals():
    assert ortho(G=None) == -1 and ortho(out=None) == -1 and ortho(G=T((6, 4), BF16, 0)) == -1
    assert ortho(G=T((6, 4), F64), out=T((6, 4), F64)) == -5 and ortho(G=T((6, 4), I8), out=T((6, 4), I8)) == -2
    assert ortho(out=T((6, 4), F32)) == -2 and ortho(out=T((4, 6), BF16)) == -3
    for shape in ((24,), (1, 1, 6, 4)):
        assert ortho(G=T(shape, BF16), out=T(shape, BF16)) == -3
    assert ortho(steps=0) == -5 and ortho(steps=-1) == -5 and ortho(steps=65) == -5
    for shape in ((65537, 4), (4, 65537), (65536, 1, 1), (60000, 4096, 4096)):
        assert ortho(G=T(shape, BF16), out=T(shape, BF16)) == -5
    assert ortho(ws=None) == -6 and ortho(n=1000) == -6 and ortho(ws=FAKE + 128) == -6
    for shape in ((0, 4), (4, 0), (0, 4, 4), (3, 4, 0)):
        assert ortho(G=T(shape, BF16), out=T(shape, BF16)) == 0
    size = om.lib().omm_orthogonalize_workspace_size
    assert size(1, 6, 4) > 0 and size(0, 6, 4) == 0 and size(1, 65537, 4) == 0 and size(1, 6, 0) == 0


def test_product_columns_of_a_launch():
    N = 2 ** 27 + 1
    wide = dict(b=T((N, 32), I8), sb=T((N,), F32), bias=None)
    assert product(Y=T((4, N), BF16), **wide) == -5
    assert product(a=T((1, 32), BF16), sa=None, Y=T((1, N), BF16), ws=FAKE, n=1 << 40, **wide) == -5
