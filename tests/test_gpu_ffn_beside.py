"""The gated block's backward pass where its slopes are computed beside the gradients' GEMM (long contractions over many
rows), against float64 and captured in a graph (needs a GB300).  Bounds: tests/ffn_ref.py."""

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


def make(W, sizes, H1, N, dt, seed):
    rng = np.random.default_rng(seed)
    e, A = len(sizes), sum(sizes)
    c = np.zeros((W, e), np.int64)
    for j, n in enumerate(sizes):
        c[:, j] = np.diff(np.concatenate([[0], np.sort(rng.integers(0, n + 1, W - 1)), [n]]))
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).to(dt)
    return (c.reshape(-1).astype(np.int32), rnd(A, H1), rnd(e, H1, N, std=H1 ** -0.5), rnd(e, H1, N, std=H1 ** -0.5),
            rnd(A, N, std=0.5))


@pytest.mark.parametrize("W,sizes,H1,N,dt,act", [
    (1, [9001], 1536, 1448, torch.bfloat16, "silu"),
    (3, [5003, 0, 17, 1, 4101], 1536, 1448, torch.float16, "gelu_tanh"),
    (2, [127, 12000, 33], 776, 2200, torch.bfloat16, "silu"),
])
def test_against_float64(W, sizes, H1, N, dt, act):
    e, A = len(sizes), sum(sizes)
    assert A * H1 * N >= 2e10
    counts, x, wg, wu, dh = make(W, sizes, H1, N, dt, 17)
    f = R.gated(x, counts, W, e, wg, wu, act)
    plan = binding.GatedPlan(W, e, A, H1, N, dt, act, save=True)
    xd, gd, ud, dd, rc = x.cuda(), wg.cuda(), wu.cuda(), dh.cuda(), torch.from_numpy(counts).cuda()
    t = plan.run(xd, rc, gd, ud)
    R.assert_rounded(t.h, f["h"], f["eh"], "h")
    b = plan.backward(dd, t.permuteOut, rc, gd, ud, t.saved)
    assert binding.a2av_gmm_read_device_status(plan.workspace) == (0, 0)
    (dx, ex), ((dg, eg), (du, eu)) = R.gated_backward(f, dh, wg, wu, act, dt)
    R.assert_rounded(b.dAtaOut, dx, ex, "dAtaOut")
    R.assert_rounded(b.dGate, dg, eg, "dGate")
    R.assert_rounded(b.dUp, du, eu, "dUp")
    # one after the other (no gradient of the rows): the same bits of the weights' gradients
    only = plan.backward(dd, t.permuteOut, rc, gd, ud, t.saved, want_rows=False)
    assert torch.equal(only.dGate.view(torch.int16), b.dGate.view(torch.int16))
    assert torch.equal(only.dUp.view(torch.int16), b.dUp.view(torch.int16))
    for _ in range(5):
        again = plan.backward(dd, t.permuteOut, rc, gd, ud, t.saved)
        for p, q in zip(again, b):
            assert torch.equal(p.view(torch.int16), q.view(torch.int16))
    # captured and replayed
    out = dict(dAtaOut=torch.zeros_like(b.dAtaOut), dGate=torch.zeros_like(b.dGate), dUp=torch.zeros_like(b.dUp))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.backward(dd, t.permuteOut, rc, gd, ud, t.saved, **out)
    for _ in range(3):
        for v in out.values():
            v.zero_()
        graph.replay()
        for k, v in out.items():
            assert torch.equal(v.view(torch.int16), getattr(b, k).view(torch.int16))
