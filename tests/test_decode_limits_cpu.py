"""Sizes past what a launch can take are refused on the host, as unsupported."""
import os
import subprocess
import sys

import pytest

om = pytest.importorskip("onnx_matmul_family_amd._omm")

from tests.test_abi_cpu import BF16, F32, I32, I64, T  # noqa: E402
from tests.test_decode_abi_cpu import layer_args, layer_call, lora_args, lora_call, lp_args, lp_call, opt, route_call  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
BLOCKS = 1 << 24  # workgroups of 256 threads: 2^32 threads, one more than a grid has


def test_rows_of_token_logprobs():
    assert lp_call(lp_args(M=BLOCKS, V=2, k=0)) == -5
    assert lp_call(lp_args(M=1 << 31, V=2, k=1)) == -5
    assert lp_call(lp_args(M=1, V=(1 << 31) - 1, k=1)) == -5


@pytest.mark.parametrize("M,V", [(BLOCKS, 2), (BLOCKS // 8, 131072), (1, (1 << 31) - 1)])
def test_rows_of_the_gradient(M, V):
    x, t, v = T((M, V), BF16), T((M,), I64), T((M,), F32)
    assert om.lib().omm_token_logprobs_grad(opt(x), opt(t), opt(v), opt(v), opt(v), opt(v), opt(x), None) == -5


def test_rows_of_the_router():
    M = 16 * BLOCKS
    assert route_call(T((M, 4), BF16), 2, T((M, 2), I32), T((M, 2), F32)) == -5


@pytest.mark.parametrize("trans", [0, 1])
def test_columns_of_the_layer(trans):
    for K, F in ((64 * BLOCKS, 1), (1, 64 * BLOCKS)):
        a = layer_args(M=1, K=K, F=F, E=2, trans=trans)
        a.update(n=1 << 62)
        assert layer_call(a) == -5


@pytest.mark.parametrize("trans", [0, 1])
def test_columns_of_the_projection(trans):
    a = lora_args(M=1, K=1, N=256 * BLOCKS, r=1, trans=trans)
    a.update(n=1 << 62)
    assert lora_call(a) == -5


@pytest.mark.parametrize("sizes", [(2, 8, 6, 4, 0), (2, 8, 0, 4, 0), (64, 4096, 2048, 512, 0),
                                   (1 << 31, 1 << 20, 256, 9, 1 << 32), (1, 1 << 62, 1 << 62, 4, 2)])
def test_workspace_of_a_layer_that_is_refused(sizes):
    """Asked for before the call's own checks: no division by the number of pairs, be it 0 or past 64 bits."""
    code = "from onnx_matmul_family_amd import _omm as om; assert om.lib().omm_moe_layer_workspace_size%r == 0" % (sizes,)
    assert subprocess.run([sys.executable, "-c", code], cwd=ROOT).returncode == 0
