"""Outputs that a caller of the C entries leaves out: the layer norm's gradient without dgamma and dbeta, its statistics one by
one, the few-token layer without the choice (needs a GB300)."""

import ctypes

import pytest
import torch

from token_permute_grouped_gb300 import binding, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()


def rnd(seed, *shape, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g).to(dtype).cuda()


def ptr(t):
    return 0 if t is None else t.data_ptr()


@pytest.mark.parametrize("rows,H", [(1, 64), (9, 2048), (61, 4096), (200, 1024), (3000, 256), (20, 9000), (5, 20000)])
def test_norm_gradient_without_the_weights(rows, H):
    dy, h, dh, gamma = rnd(1, rows, H), rnd(2, rows, H), rnd(3, rows, H), rnd(4, H)
    mean, rstd = rnd(5, rows, dtype=torch.float32), rnd(6, rows, dtype=torch.float32).abs()
    want, _, _ = binding.a2av_layer_norm_backward(dy, h, gamma, mean, rstd, dh)
    dx = torch.empty_like(dy)
    stream = torch.cuda.current_stream().cuda_stream
    args = [ptr(t) for t in (dy, dh, h, gamma, mean, rstd, dx, None, None, None)]
    for _ in range(2):
        assert binding.load().a2av_layer_norm_backward(rows, H, binding.DTYPES[torch.bfloat16], *args, 0, stream) == 0
    torch.cuda.synchronize()
    assert torch.equal(dx.view(torch.int16), want.view(torch.int16))


@pytest.mark.parametrize("rows,H", [(1, 64), (300, 4096), (700, 2048), (3, 20000)])
def test_norm_with_one_output_at_a_time(rows, H):
    x, res, gamma, beta = rnd(7, rows, H), rnd(8, rows, H), rnd(9, H), rnd(10, H)
    whole = binding.a2av_layer_norm(x, gamma, beta, res, want_y=True, want_stats=True)
    desc = ctypes.byref(binding.LayerNormDesc(rows, H, H, H, binding.DTYPES[torch.bfloat16], -1, 0, 1e-5))
    for name in ("h", "y", "mean", "rstd"):
        want = getattr(whole, name)
        got = torch.full_like(want, 7.0)
        outs = [ptr(got) if n == name else 0 for n in ("h", "y")] + [0, 0] + [ptr(got) if n == name else 0 for n in ("mean", "rstd")]
        stream = torch.cuda.current_stream().cuda_stream
        assert binding.load().a2av_layer_norm(desc, ptr(x), ptr(res), ptr(gamma), ptr(beta), *outs, stream) == 0
        torch.cuda.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("T", [1, 7, 40])
def test_few_token_layer_without_the_choice(T):
    E, K, H, N = 12, 3, 264, 136
    x, router, gate, up, down = (rnd(11 + i, *s) for i, s in enumerate(((T, H), (E, H), (E, H, N), (E, H, N), (E, N, H))))
    plan = binding.MoePlan(T, E, K, H, N)
    want = plan.run(x, router, gate, up, down)
    for outs in ((None, None), (torch.empty_like(want.experts), None), (None, torch.empty_like(want.weights))):
        y = torch.empty_like(x)
        stream = torch.cuda.current_stream().cuda_stream
        args = [ptr(t) for t in (x, router, None, gate, up, down, None, y, *outs, plan.workspace)]
        assert binding.load().a2av_moe_run(ctypes.byref(plan.desc), *args, plan.workspace.numel(), stream) == 0
        torch.cuda.synchronize()
        assert torch.equal(y, want.y)
        assert outs[0] is None or torch.equal(outs[0], want.experts)
        assert outs[1] is None or torch.equal(outs[1], want.weights)
