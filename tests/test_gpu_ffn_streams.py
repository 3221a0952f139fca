"""Tensors that the expert-layer calls make for themselves belong to the stream that works on them: memory the caller's
own stream has freed but may still be reading is not written, and a call's workspace is not handed out while the call is
still running (needs a GB300)."""

import pytest
import torch

from token_permute_grouped_gb300 import binding, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()


def freed(*sizes):
    """Addresses of blocks of these sizes that the current stream has used and given back."""
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]
    at = {b.data_ptr() for b in blocks}
    del blocks
    return at


def rnd(*shape):
    return torch.randn(*shape, device="cuda").bfloat16()


def calls():
    rows, H, W, e, N = 400, 1024, 2, 2, 256
    x, dy, gamma = rnd(rows, H), rnd(rows, H), rnd(H)
    rstd = torch.rand(rows, device="cuda")
    gu = rnd(rows, 2 * N)
    rc = torch.tensor([100, 100, 100, 100], dtype=torch.int32, device="cuda")
    wg, wu, wd = rnd(e, H, N), rnd(e, H, N), rnd(e, H, N)
    plan = binding.GatedPlan(W, e, rows, H, N, save=True)
    kept = plan.run(x, rc, wg, wu)
    dh = rnd(rows, N)
    gmm = binding.GmmBackwardPlan(W, e, rows, H, N)
    return {
        "norm": lambda s: binding.a2av_rms_norm(x, gamma, dy, 1e-6, "e4m3fn", "mx", True, True, stream=s),
        "norm_backward": lambda s: binding.a2av_rms_norm_backward(dy, x, gamma, rstd, stream=s),
        "glu": lambda s: binding.a2av_glu_quant(gu, want_h=True, stream=s),
        "gated": lambda s: plan.run(x, rc, wg, wu, stream=s),
        "gated_backward": lambda s: plan.backward(dh, kept.permuteOut, rc, wg, wu, kept.saved, stream=s),
        "gmm_backward": lambda s: gmm.run(dh, kept.permuteOut, rc, wd, stream=s),
    }


@pytest.mark.parametrize("name", ["norm", "norm_backward", "glu", "gated", "gated_backward", "gmm_backward"])
def test_outputs_are_of_the_stream_that_writes_them(name):
    call = calls()[name]
    first = [t for t in call(None) if t is not None]
    sizes = [t.numel() * t.element_size() for t in first]
    torch.cuda.synchronize()
    mine = freed(*sizes)
    s = torch.cuda.Stream()
    got = [t for t in call(s) if t is not None]
    torch.cuda.synchronize()
    assert not mine & {t.data_ptr() for t in got}
    for a, b in zip(first, got):
        assert torch.equal(a, b)


def test_workspace_is_not_given_away_while_the_call_runs(monkeypatch):
    rows, H = 400, 1024
    dy, h, gamma, rstd = rnd(rows, H), rnd(rows, H), rnd(H), torch.rand(rows, device="cuda")
    seen = []
    plain = binding._call
    monkeypatch.setattr(binding, "_call", lambda name, *a: (seen.append((name, a)), plain(name, *a))[1])
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = binding.a2av_rms_norm_backward(dy, h, gamma, rstd, stream=s)
    at, need = [a[-3:-1] for n, a in seen if n == "a2av_rms_norm_backward"][0]
    assert need > 0
    after = [torch.empty(need, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert at not in {t.data_ptr() for t in after}
    torch.cuda.synchronize()
    assert bool(torch.isfinite(out[1]).all())
