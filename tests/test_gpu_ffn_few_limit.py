"""The gated block on both sides of the numbers of rows at which another kernel takes the call, with even and with skewed
routing, against float64 (on the GPU).  Bounds: tests/ffn_ref.py."""

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


@pytest.mark.parametrize("W,H1,N,sizes", [
    (1, 4096, 264, [72, 72]), (3, 4096, 264, [80, 80]), (2, 4096, 264, [140, 4]), (2, 4096, 136, [160, 0]),
    (2, 4104, 136, [129, 131]), (1, 4096, 136, [255]), (1, 4096, 136, [257]), (4, 1032, 328, [41, 43, 38]),
    (4, 1032, 328, [48, 52, 51]), (2, 1032, 328, [120, 0, 0]),
])
@pytest.mark.parametrize("save", [False, True])
def test_gated(W, H1, N, sizes, save):
    e, A, dt = len(sizes), sum(sizes), torch.bfloat16
    rng = np.random.default_rng(6)
    counts = np.zeros((W, e), np.int64)
    for j, n in enumerate(sizes):
        counts[:, j] = np.diff(np.concatenate([[0], np.sort(rng.integers(0, n + 1, W - 1)), [n]]))
    counts = counts.reshape(-1).astype(np.int32)
    g = torch.Generator().manual_seed(6)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(dt)
    x, wg, wu = rnd(A, H1), rnd(e, H1, N, std=H1 ** -0.5), rnd(e, H1, N, std=H1 ** -0.5)
    f = R.gated(x, counts, W, e, wg, wu, "silu")
    plan = binding.GatedPlan(W, e, A, H1, N, dt, save=save)
    r = plan.run(x.cuda(), torch.from_numpy(counts).cuda(), wg.cuda(), wu.cuda())
    assert binding.a2av_gmm_read_device_status(plan.workspace) == (0, 0)
    R.assert_rounded(r.h, f["h"], f["eh"], "h")
    if save:
        assert torch.equal(r.permuteOut.cpu().view(torch.int16), x[f["idx"]].view(torch.int16))
        for got, ref, err in ((r.saved[0], f["G"], f["eg"]), (r.saved[1], f["U"], f["eu"])):
            assert bool(((got.cpu().double() - ref).abs() <= err).all())
