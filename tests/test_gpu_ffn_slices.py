"""Gradients whose contraction is cut into slices (few tiles over long contractions), against float64 (needs a GB300).
Bounds: tests/ffn_ref.py."""

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


def make(W, H1, N, sizes, dt, seed):
    rng = np.random.default_rng(seed)
    e, A = len(sizes), sum(sizes)
    c = np.zeros((W, e), np.int64)
    for j, n in enumerate(sizes):
        c[:, j] = np.diff(np.concatenate([[0], np.sort(rng.integers(0, n + 1, W - 1)), [n]]))
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(dt)
    return (e, A, c.reshape(-1).astype(np.int32), rnd(A, H1), rnd(e, H1, N, std=H1 ** -0.5),
            rnd(e, H1, N, std=H1 ** -0.5), rnd(A, N, std=0.5))


# W, H1, N, rows of each expert: sliced along an expert's rows; experts with fewer rows than there are slices, or
# none; along wide rows of few tokens; along both.
SHAPES = [
    (1, 64, 72, [3000]),
    (2, 200, 136, [9000, 0, 1, 130, 2049]),
    (4, 448, 256, [9000, 15]),
    (1, 136, 3400, [1, 2]),
    (3, 264, 2056, [40, 0, 7]),
    (2, 128, 2048, [900]),
]


@pytest.mark.parametrize("W,H1,N,sizes", SHAPES)
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_grouped_product(W, H1, N, sizes, dt):
    e, A, counts, x, w, _, dy = make(W, H1, N, sizes, dt, 7)
    idx, _ = R.arrival_index(counts, W, e)
    plan = binding.GmmBackwardPlan(W, e, A, H1, N, dt)
    assert plan.workspace.numel() > 256  # the slices' sums
    args = [t.cuda() for t in (dy, x[idx], torch.from_numpy(counts), w)]
    dx, dw = plan.run(*args)
    assert binding.a2av_gmm_read_device_status(plan.workspace) == (0, 0)
    (rx, ex), ((rw, ew),) = R.gmm_backward(x[idx], counts, W, e, dy, w)
    R.assert_rounded(dx, rx, ex, "dAtaOut")
    R.assert_rounded(dw, rw, ew, "dWeight")
    for _ in range(3):  # the same bits, together and alone
        again = plan.run(*args)
        assert torch.equal(again[0].view(torch.int16), dx.view(torch.int16))
        assert torch.equal(again[1].view(torch.int16), dw.view(torch.int16))
    assert torch.equal(plan.run(*args, want_weights=False)[0].view(torch.int16), dx.view(torch.int16))
    assert torch.equal(plan.run(*args, want_rows=False)[1].view(torch.int16), dw.view(torch.int16))


@pytest.mark.parametrize("W,H1,N,sizes", SHAPES + [(1, 128, 264, [9000])])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated(W, H1, N, sizes, act, dt=torch.bfloat16):
    e, A, counts, x, wg, wu, dh = make(W, H1, N, sizes, dt, 11)
    f = R.gated(x, counts, W, e, wg, wu, act)
    plan = binding.GatedPlan(W, e, A, H1, N, dt, act, save=True)
    xd, gd, ud, dd, rc = x.cuda(), wg.cuda(), wu.cuda(), dh.cuda(), torch.from_numpy(counts).cuda()
    t = plan.run(xd, rc, gd, ud)
    b = plan.backward(dd, t.permuteOut, rc, gd, ud, t.saved)
    assert binding.a2av_gmm_read_device_status(plan.workspace) == (0, 0)
    (dx, ex), ((dg, eg), (du, eu)) = R.gated_backward(f, dh, wg, wu, act, dt)
    R.assert_rounded(b.dAtaOut, dx, ex, "dAtaOut")
    R.assert_rounded(b.dGate, dg, eg, "dGate")
    R.assert_rounded(b.dUp, du, eu, "dUp")


def test_not_finite_rows_stay_in_their_expert():
    W, H1, N, sizes = 2, 200, 136, [4700, 45, 4900]
    e, A, counts, x, w, _, dy = make(W, H1, N, sizes, torch.bfloat16, 3)
    idx, _ = R.arrival_index(counts, W, e)
    plan = binding.GmmBackwardPlan(W, e, A, H1, N)
    assert plan.workspace.numel() > 256
    rc, wd, xe = torch.from_numpy(counts).cuda(), w.cuda(), x[idx].cuda()
    good = plan.run(dy.cuda(), xe, rc, wd)[1].cpu()
    for bad in (float("inf"), float("nan")):
        xb, yb = xe.clone(), dy.clone()
        xb[4700:4745] = bad
        yb[4700:4745] = bad
        dw = plan.run(yb.cuda(), xb, rc, wd)[1].cpu()
        assert torch.equal(dw[[0, 2]].view(torch.int16), good[[0, 2]].view(torch.int16))
        assert not bool(torch.isfinite(dw[1].float()).all())


def test_inconsistent_counts_write_nothing():
    W, H1, N, sizes = 2, 64, 72, [1500, 1600]
    e, A, counts, x, w, _, dy = make(W, H1, N, sizes, torch.bfloat16, 5)
    plan = binding.GmmBackwardPlan(W, e, A, H1, N)
    assert plan.workspace.numel() > 256
    rc = torch.from_numpy(counts).cuda()
    rc[1] += 1
    dx = torch.full((A, H1), 7.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((e, H1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    plan.run(dy.cuda(), x.cuda(), rc, w.cuda(), dAtaOut=dx, dWeight=dw)
    status = binding.a2av_gmm_read_device_status(plan.workspace)
    assert binding.STATUS_NAMES[status[0]] == "A2AV_ERR_DEVICE_CHECK"
    assert bool((dx == 7.0).all()) and bool((dw == 7.0).all())
