"""Every kernel that int8_matmul and orthogonalize choose between, against the definitions, and that these sizes
choose it."""
import os
import subprocess
import sys

import pytest
import torch

from tests.decode_util import TORCH, assert_within
from tests.test_gpu_orthogonalize import draw
from tests.train_util import int8_product, orthogonalise, orthogonalise_tol

pytestmark = pytest.mark.gpu

om = pytest.importorskip("onnx_matmul_family_amd._omm")

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# (M, K, N): what an int8 a takes, what a bf16 a takes where that differs
PRODUCTS = {
    (4, 528, 4000): ("streamed, 16 x 16 a workgroup, 4 units",),
    (4, 528, 6150): ("streamed, 16 x 16 a workgroup, 2 units",),
    (12, 272, 8300): ("streamed, 16 x 32 a workgroup, 2 units",),
    (2, 1040, 8300): ("streamed, 16 x 32 a workgroup, 2 units", "streamed, 16 x 32 a workgroup, 2 units at once, quantised"),
    (1, 515, 8000): ("streamed, 16 x 16 a workgroup, 2 units", "streamed, 16 x 16 a workgroup, 4 units at once, quantised"),
    (30, 400, 1003): ("streamed, 32 x 16 a workgroup, 2 units",),
    (24, 400, 5003): ("streamed, 32 x 32 a workgroup, 1 units",),
    (50, 1040, 4000): ("streamed, 64 x 16 a workgroup, 1 units",),
    (43, 4096, 4104): ("streamed, 64 x 32 a workgroup, 1 units",),
    (130, 256, 300): ("tiles of 64, two groups of waves\n",),
    (130, 272, 300): ("tiles of 64, two groups of waves, ragged\n",),
    (130, 256, 8000): ("tiles of 64\n",),
    (130, 272, 8000): ("tiles of 64, ragged\n",),
    (600, 256, 3500): ("tiles of 128, two groups of waves\n",),
    (1024, 4096, 4096): ("tiles of 128, two groups of waves\n",),
    (600, 272, 3500): ("tiles of 128, two groups of waves, ragged\n",),
    (1000, 1000, 4096): ("tiles of 128, two groups of waves, ragged\n",),
    (1100, 256, 4000): ("tiles of 128\n",),
    (1100, 272, 4000): ("tiles of 128, ragged\n",),
    (3500, 1024, 3500): ("tiles of 256\n",),
    (3584, 1024, 3584): ("tiles of 256\n",),
    (3500, 528, 3500): ("tiles of 256, ragged\n",),
    (3584, 528, 3585): ("tiles of 256, ragged\n",),
}
# (batch, m, n): tiles of A = X X^T and workgroups each, of B = aI + bA + cA^2, of B X
UPDATES = {
    (1, 520, 320): (32, 1, 32, 64),
    (1, 96, 2000): (32, 4, 32, 64),
    (18, 3200, 192): (64, 2, 64, 128),
    (1, 320, 5000): (64, 16, 32, 64),
    (1, 1440, 720): (64, 2, 64, 64),
    (12, 520, 320): (64, 1, 64, 128),
    (6, 720, 920): (64, 1, 64, 192),
    (6, 920, 720): (64, 1, 64, 192),
    (11, 680, 980): (128, 1, 128, 256),
    (11, 980, 680): (128, 1, 128, 256),
    (6, 1120, 1120): (192, 1, 192, 128),
    (14, 1160, 1160): (256, 1, 256, 256),
    (14, 1170, 1160): (256, 1, 256, 256),
}

CHILD = """
import sys, torch
sys.path.insert(0, %r)
import onnx_matmul_family_amd as omm
products, updates = %r, %r
def mark(s):
    print(s, file=sys.stderr, flush=True)
for M, K, N in products:
    W, s = torch.zeros((N, K), dtype=torch.int8, device="cuda"), torch.ones((N,), device="cuda")
    for a, sa in ((torch.zeros((M, K), dtype=torch.int8, device="cuda"), torch.ones((M,), device="cuda")),
                  (torch.zeros((M, K), dtype=torch.bfloat16, device="cuda"), None)):
        mark("case")
        omm.int8_matmul(a, W, s, a_scale=sa)
        torch.cuda.synchronize()
for Z, m, n in updates:
    mark("case")
    omm.orthogonalize(torch.zeros((Z, m, n), device="cuda"), steps=1)
    torch.cuda.synchronize()
mark("case")
"""


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    om.lib()


@pytest.fixture(scope="module")
def choices(_gpu):
    """What a process that logs its choices prints, a text for each call above."""
    r = subprocess.run([sys.executable, "-c", CHILD % (ROOT, list(PRODUCTS), list(UPDATES))], capture_output=True,
                       text=True, timeout=100, env=dict(os.environ, OMM_LOG="1"))
    assert r.returncode == 0, r.stderr[-2000:]
    parts = r.stderr.split("case\n")[1:-1]
    products = {c: parts[2 * i:2 * i + 2] for i, c in enumerate(PRODUCTS)}
    updates = {c: parts[2 * len(PRODUCTS) + i] for i, c in enumerate(UPDATES)}
    return products, updates


@pytest.mark.parametrize("case", list(PRODUCTS), ids=str)
def test_choice_of_a_product(choices, case):
    want = PRODUCTS[case]
    for text, part in zip(choices[0][case], (want[0], want[-1])):
        assert text.count("omm: int8_matmul") == 1 and part in text, (part, text)


@pytest.mark.parametrize("case", list(UPDATES), ids=str)
def test_choice_of_an_update(choices, case):
    lines = [x for x in choices[1][case].splitlines() if x.startswith("omm: orthogonalize")]
    got = [[int(v) for v in x.split("tiles of ")[1].split(" workgroups")[0].split(", ")] for x in lines]
    a, split, b, u = UPDATES[case]
    assert got == [[a, split], [b, 1], [u, 1]]


@pytest.mark.parametrize("case", list(PRODUCTS), ids=str)
@pytest.mark.parametrize("dt,bias", [("bf16", False), ("f16", True), ("f32", True)])
def test_product(case, dt, bias):
    """The definition on the GPU, in 64 bits, by a library product (of integers below 2^53: exact)."""
    M, K, N = case
    gen = torch.Generator(device="cuda").manual_seed(M + K + N)
    X = torch.randn((M, K), generator=gen, device="cuda").to(TORCH[dt])
    W = torch.randint(-128, 128, (N, K), generator=gen, device="cuda", dtype=torch.int8)
    sb = torch.rand((N,), generator=gen, device="cuda") * 0.02 + 1e-4
    b = torch.randn((N,), generator=gen, device="cuda").to(TORCH[dt]) if bias else None
    q, sa = om.quantize_rows(X)  # (tested by itself)
    want, tol = int8_product(q, sa, W, sb, b, dt)
    got = om.int8_matmul(q, W, sb, a_scale=sa, bias=b, dtype=X.dtype)[0]
    assert_within(got, want.cpu(), tol.cpu(), "int8 rows")
    assert torch.equal(om.int8_matmul(X, W, sb, bias=b)[0], got)


@pytest.mark.parametrize("case", list(UPDATES), ids=str)
@pytest.mark.parametrize("dt", ["bf16", "f16", "f32"])
def test_update(case, dt):
    Z, m, n = case
    G = torch.stack([draw(m, n, dt, rank=3, seed=z) for z in range(Z)])
    got, _ = om.orthogonalize(G.cuda())
    for z in sorted({0, Z - 1}):
        want = orthogonalise(G[z].cuda(), 5)
        assert_within(got[z], want.cpu(), orthogonalise_tol(G[z].cuda(), want, 5, dt).cpu(), "%d of %d" % (z, Z))
    # alone, by whatever tiles that takes: the sums' order differs, no more
    alone, _ = om.orthogonalize(G[1 if Z > 1 else 0].cuda())
    want = orthogonalise(G[1 if Z > 1 else 0].cuda(), 5)
    tol = orthogonalise_tol(G[1 if Z > 1 else 0].cuda(), want, 5, dt)
    assert_within(alone, want.cpu(), tol.cpu(), "alone")
