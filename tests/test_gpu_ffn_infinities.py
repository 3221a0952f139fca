"""Infinities in an operand of the gated block's gradients, for a few rows and for more, against the float64 formula: an
infinite weight or input gives an infinity where the formula does (on the GPU).  Bounds: tests/ffn_ref.py."""

import pytest
import torch

import ffn_ref as R
from token_permute_grouped_gb300 import binding, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()


@pytest.mark.parametrize("A", [1, 20, 32, 33, 70])
@pytest.mark.parametrize("where", ["gate", "up", "x", "dh"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_an_infinity_stays_one(A, where, dt):
    H1, N, name = 64, 96, "silu"
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g)
    x, wg, wu, dh = rnd(A, H1).to(dt), rnd(1, H1, N).to(dt), rnd(1, H1, N).to(dt), rnd(A, N).to(dt)
    G, U = rnd(A, N), rnd(A, N)
    # Slopes that are 16-bit numbers already: nothing is left over of their rounding.
    G[:, ::4] = 0.0                                   # dG = dh U / 2, dU = 0
    U[:, ::4] = torch.where(U[:, ::4] < 0, -0.5, 2.0)
    inf = float("inf")
    if where == "gate":
        wg[0, 5, 8], wg[0, 9, 3] = inf, -inf          # of a column with such slopes, and of another
    elif where == "up":
        wu[0, 5, 7], wu[0, 9, 3] = inf, -inf
    elif where == "x":
        x[0, 5], x[A - 1, 9] = inf, -inf
    else:
        dh[0, 8] = inf
    f = {"xe": x.double(), "sizes": [A], "idx": torch.arange(A), "G": G.double(), "U": U.double(),
         "eg": torch.zeros(A, N).double(), "eu": torch.zeros(A, N).double()}
    (dx, ex), ((dg, eg), (du, eu)) = R.gated_backward(f, dh, wg, wu, name, dt)
    plan = binding.GatedPlan(1, 1, A, H1, N, dt, name, save=True)
    rc = torch.tensor([A], dtype=torch.int32, device="cuda")
    b = plan.backward(dh.cuda(), x.cuda(), rc, wg.cuda(), wu.cuda(), torch.stack([G, U]).cuda())
    assert not bool(torch.isfinite(dx).all() and torch.isfinite(dg).all())
    for got, ref, err, what in ((b.dAtaOut, dx, ex, "dAtaOut"), (b.dGate, dg, eg, "dGate"), (b.dUp, du, eu, "dUp")):
        got = got.cpu().double()
        gone = torch.isinf(ref)
        assert torch.equal(torch.isnan(got), torch.isnan(ref)), what
        assert bool((got == ref)[gone].all()), what
        fine = torch.isfinite(ref)
        R.assert_rounded(got[fine].to(dt), ref[fine], err[fine], what)
