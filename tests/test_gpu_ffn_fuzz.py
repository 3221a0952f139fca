"""Seeded random shapes of the gated block, its backward pass and the grouped product's gradients against float64 (needs
a GB300): widths that are and are not multiples of 64 and 128, empty experts, one row to a few hundred an expert, one
source to many, so that every tile shape, row pass and split of the kernels is met.  Bounds: tests/ffn_ref.py."""

import numpy as np
import pytest
import torch

import ffn_ref as R
from token_permute_grouped_gb300 import binding, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()


def draw(seed):
    rng = np.random.default_rng(seed)
    e, W = int(rng.choice([1, 2, 3, 7, 16])), int(rng.choice([1, 1, 2, 5, 16]))
    step = int(rng.choice([8, 64, 128]))
    wide = int(rng.choice([200, 700, 2100 if e < 4 else 700]))
    H1 = max(8, int(rng.integers(1, wide // step + 1)) * step)
    N = max(8, int(rng.integers(1, 700 // step + 1)) * step)
    top = int(rng.choice([3, 20, 70, 140, 300]))
    counts = rng.integers(0, top // W + 2, W * e)
    counts[rng.random(W * e) < rng.choice([0.0, 0.3])] = 0
    if counts.sum() == 0:
        counts[0] = 1
    dt = torch.bfloat16 if rng.random() < 0.5 else torch.float16
    return W, e, H1, N, counts.astype(np.int32), dt, str(rng.choice(["silu", "gelu_tanh"]))


@pytest.mark.parametrize("seed", range(48))
def test_random_shape(seed):
    W, e, H1, N, counts, dt, act = draw(seed)
    A = int(counts.sum())
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(dt)
    x, wg, wu, dh = rnd(A, H1), rnd(e, H1, N, std=H1 ** -0.5), rnd(e, H1, N, std=H1 ** -0.5), rnd(A, N, std=0.5)
    xd, gd, ud, dd, rc = x.cuda(), wg.cuda(), wu.cuda(), dh.cuda(), torch.from_numpy(counts).cuda()
    f = R.gated(x, counts, W, e, wg, wu, act)
    serve = binding.GatedPlan(W, e, A, H1, N, dt, act)
    R.assert_rounded(serve.run(xd, rc, gd, ud).h, f["h"], f["eh"], "h")
    plan = binding.GatedPlan(W, e, A, H1, N, dt, act, save=True)
    t = plan.run(xd, rc, gd, ud)
    R.assert_rounded(t.h, f["h"], f["eh"], "h (kept)")
    assert torch.equal(t.permuteOut.cpu().view(torch.int16), x[f["idx"]].view(torch.int16))
    b = plan.backward(dd, t.permuteOut, rc, gd, ud, t.saved)
    (dx, ex), ((dg, eg), (du, eu)) = R.gated_backward(f, dh, wg, wu, act, dt)
    R.assert_rounded(b.dAtaOut, dx, ex, "dAtaOut")
    R.assert_rounded(b.dGate, dg, eg, "dGate")
    R.assert_rounded(b.dUp, du, eu, "dUp")
    m = binding.GmmBackwardPlan(W, e, A, H1, N, dt)
    mx, mw = m.run(dd, t.permuteOut, rc, gd)
    (rx, ex), ((rw, ew),) = R.gmm_backward(x[f["idx"]], counts, W, e, dh, wg)
    R.assert_rounded(mx, rx, ex, "gmm dAtaOut")
    R.assert_rounded(mw, rw, ew, "gmm dWeight")
    for q in (serve, plan, m):
        assert binding.a2av_gmm_read_device_status(q.workspace) == (0, 0)
