"""How far the gated block's gradients are from float64 on either side of the number of rows up to which the slopes are kept
in two summands: the error of one rounding, or of two independent ones (on the GPU)."""

import pytest
import torch

import ffn_ref as R
from token_permute_grouped_gb300 import binding, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("sizes,roundings", [
    ([1] * 32, 1), ([2] + [1] * 31, 2),   # many experts of one row
    ([32], 1), ([33], 2), ([400], 2),
])
def test_error(sizes, roundings, dt):
    e, A, H1, N = len(sizes), sum(sizes), 256, 192
    g = torch.Generator().manual_seed(4)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(dt)
    x, dh = rnd(A, H1), rnd(A, N)
    wg, wu = rnd(e, H1, N, std=H1 ** -0.5), rnd(e, H1, N, std=H1 ** -0.5)
    f = R.gated(x, sizes, 1, e, wg, wu, "silu")
    (dx, _), ((dg, _), (du, _)) = R.gated_backward(f, dh, wg, wu, "silu", dt)
    plan = binding.GatedPlan(1, e, A, H1, N, dt, save=True)
    rc = torch.tensor(sizes, dtype=torch.int32, device="cuda")
    xd, gd, ud = x.cuda(), wg.cuda(), wu.cuda()
    t = plan.run(xd, rc, gd, ud)
    b = plan.backward(dh.cuda(), t.permuteOut, rc, gd, ud, t.saved)
    for got, ref in ((b.dAtaOut, dx), (b.dGate, dg), (b.dUp, du)):
        one = float((ref.to(dt).double() - ref).norm())
        off = float((got.cpu().double() - ref).norm())
        # (two roundings of equal, independent errors; a tenth for chance)
        assert off <= 1.1 * roundings ** 0.5 * one, (off / one)
