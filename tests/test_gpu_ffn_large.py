"""The expert-layer operators on tensors whose offsets pass 2^31 elements, on sampled rows against float64 (on the GPU).
Bounds as in tests/ffn_ref.py."""

import pytest
import torch

import ffn_ref as R
from token_permute_grouped_gb300 import binding, build

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    yield
    torch.cuda.empty_cache()


def filled(*shape, seed, std=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return torch.empty(*shape, dtype=torch.bfloat16, device=DEV).normal_(0.0, std, generator=g)


def sample(rows):
    return torch.tensor([0, 1, 2 ** 18 - 1, 2 ** 18, rows // 2, rows - 2, rows - 1], device=DEV)


def test_norm_and_its_gradient():
    rows, H = 2 ** 18 + 1001, 8192  # 2.16e9 values
    x, gamma = filled(rows, H, seed=1), filled(H, seed=2)
    r = binding.a2av_rms_norm(x, gamma, None, 1e-6, "e4m3fn", "mx", want_y=True, want_rstd=True)
    at = sample(rows)
    s, y, _ = R.rms_norm(x[at].cpu(), None, gamma.cpu(), 1e-6)
    R.assert_rounded(r.y[at], y, y.abs() * R.CHAIN, "y")
    R.assert_codes(r.codes[at], r.scales[at], y, R.CHAIN, "e4m3fn", "mx", "codes")
    dx, dgamma = binding.a2av_rms_norm_backward(r.y, x, gamma, r.rstd)
    h, dy, rstd = x[at].cpu(), r.y[at].cpu(), r.rstd[at].cpu()
    ref, _ = R.rms_norm_backward(dy, None, h, gamma.cpu(), rstd)
    n, a = h.double() * rstd.double()[:, None], dy.double() * gamma.cpu().double()
    err = R.CHAIN * rstd.double()[:, None] * (a.abs() + n.abs() * (a * n).abs().mean(1, keepdim=True)) + 2.0 ** -23 * ref.abs()
    R.assert_rounded(dx[at], ref, err, "dx")
    cols = slice(8000, 8064)
    nd = x[:, cols].double() * r.rstd.double()[:, None] * r.y[:, cols].double()
    assert bool(((dgamma[cols].double() - nd.sum(0)).abs() <= nd.abs().sum(0) * 1e-5).all())


def test_glu_quant():
    rows, N = 2 ** 18 + 1001, 4096  # 2.16e9 values in, 1.08e9 codes out
    gu = filled(rows, 2 * N, seed=3)
    r = binding.a2av_glu_quant(gu, "silu", "e5m2", "group128", want_h=True)
    at = sample(rows)
    z = gu[at].cpu().double()
    v = R.act(z[:, :N], "silu") * z[:, N:]
    R.assert_rounded(r.h[at], v, v.abs() * R.CHAIN, "h")
    R.assert_codes(r.codes[at], r.scales[at], v, R.CHAIN, "e5m2", "group128", "codes")


@pytest.mark.parametrize("H1", [64, 1024])  # slopes before the gradients' GEMM; beside it
def test_gated_block(H1):
    W, e, N = 3, 2, 2048
    A = 540_000  # saved: 2.2e9 values
    counts = torch.tensor([150_000, 70_001, 1, 199_998, 100_000, 20_000], dtype=torch.int32)
    assert int(counts.sum()) == A
    x, dh = filled(A, H1, seed=5), filled(A, N, seed=6, std=0.5)
    wg, wu = filled(e, H1, N, seed=7, std=H1 ** -0.5), filled(e, H1, N, seed=8, std=H1 ** -0.5)
    rc = counts.to(DEV)
    plan = binding.GatedPlan(W, e, A, H1, N, save=True)
    t = plan.run(x, rc, wg, wu)
    b = plan.backward(dh, t.permuteOut, rc, wg, wu, t.saved)
    assert binding.a2av_gmm_read_device_status(plan.workspace) == (0, 0)
    idx, sizes = R.arrival_index(counts.tolist(), W, e)
    pick = torch.tensor([0, 1, sizes[0] - 1, sizes[0], A // 2, A - 2, A - 1])
    expert = (pick >= sizes[0]).long()
    xs = x[idx[pick].to(DEV)].cpu()
    for k in range(len(pick)):  # one row at a time: a one-row problem of its expert
        j = int(expert[k])
        w1, w2 = wg[j:j + 1].cpu(), wu[j:j + 1].cpu()
        f = R.gated(xs[k:k + 1], [1], 1, 1, w1, w2, "silu")
        R.assert_rounded(t.h[pick[k]:pick[k] + 1], f["h"], f["eh"], "h")
        assert bool(((t.saved[0, pick[k]].cpu().double() - f["G"][0]).abs() <= f["eg"][0]).all())
        assert bool(((t.saved[1, pick[k]].cpu().double() - f["U"][0]).abs() <= f["eu"][0]).all())
        (dx, ex), _ = R.gated_backward(f, dh[pick[k]:pick[k] + 1].cpu(), w1, w2, "silu", torch.bfloat16)
        R.assert_rounded(b.dAtaOut[idx[pick[k]]:idx[pick[k]] + 1], dx, ex, "dAtaOut")
    # the weights' gradient of the last expert, some columns, summed over all of its rows
    cols = slice(2000, 2032)
    G, U = t.saved[0, sizes[0]:, cols].double(), t.saved[1, sizes[0]:, cols].double()
    dG = dh[sizes[0]:, cols].double() * U * R.act_slope(G, "silu")
    xe = t.permuteOut[sizes[0]:].double()
    ref = xe.t() @ dG
    lim = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + (sizes[1] + 8) * 2.0 ** -23) * (xe.abs().t() @ dG.abs())
    assert bool(((b.dGate[1, :, cols].double() - ref).abs() <= lim).all())


def test_staged_rows():
    W, e, H1, N = 3, 2, 16384, 64
    A = 140_000  # 2.3e9 values
    counts = torch.tensor([30_000, 20_001, 1, 49_998, 25_000, 15_000], dtype=torch.int32)
    assert int(counts.sum()) == A
    x, wg, wu = filled(A, H1, seed=9), filled(e, H1, N, seed=10, std=H1 ** -0.5), filled(e, H1, N, seed=11, std=H1 ** -0.5)
    plan = binding.GatedPlan(W, e, A, H1, N, save=True)
    t = plan.run(x, counts.to(DEV), wg, wu)
    assert binding.a2av_gmm_read_device_status(plan.workspace) == (0, 0)
    idx, sizes = R.arrival_index(counts.tolist(), W, e)
    for i in range(0, A, 10_000):
        part = x[idx[i:i + 10_000].to(DEV)]
        assert torch.equal(t.permuteOut[i:i + 10_000].view(torch.int16), part.view(torch.int16))
    for k in (0, sizes[0] - 1, sizes[0], A - 1):
        j = int(k >= sizes[0])
        f = R.gated(x[idx[k]:idx[k] + 1].cpu(), [1], 1, 1, wg[j:j + 1].cpu(), wu[j:j + 1].cpu(), "silu")
        R.assert_rounded(t.h[k:k + 1], f["h"], f["eh"], "h")
