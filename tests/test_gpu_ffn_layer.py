"""The expert layer put together from the operators (token_permute_grouped_gb300/ffn.py), on the GPU against float64.

Errors are compared in the 2-norm.  bf16 path: every tensor that is rounded on the way (normed rows, h, dh, dG, dU,
and the output) adds at most u = 2^-8 of its own size, which a product carries on in proportion; with at most five
roundings behind any output the bound is 5 u.  mx path: a value's code is within 2^-4 of it (three mantissa bits; a
block's largest values, above 448 of the scaled 512, saturate by at most 1/8), so an operand is at most 2^-3 off, in
the mean far less; four operands stand behind the output: the bound is 2^-2."""

import numpy as np
import pytest
import torch

import ffn_ref as R
from token_permute_grouped_gb300 import binding, build, ffn
from token_permute_grouped_gb300.workloads import mx_quantize

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()


def _norm2(got, ref):
    return float((got.double().cpu() - ref).norm() / ref.norm())


@pytest.mark.parametrize("W,e,T,H,N,act", [(1, 4, 300, 256, 192, "silu"), (4, 3, 700, 520, 328, "gelu_tanh")])
def test_training_step(W, e, T, H, N, act):
    """Tokens -> norm with residual -> rows of the experts -> block -> gradients of everything."""
    g = torch.Generator().manual_seed(5)
    rnd = lambda *s, std=1.0: (torch.randn(*s, generator=g) * std).bfloat16()
    x, res, gamma = rnd(T, H), rnd(T, H, std=2.0), (1 + 0.1 * torch.randn(H, generator=g)).bfloat16()
    gate, up, down = rnd(e, H, N, std=H ** -0.5), rnd(e, H, N, std=H ** -0.5), rnd(e, N, H, std=N ** -0.5)
    counts = np.random.default_rng(3).multinomial(T, np.ones(W * e) / (W * e)).astype(np.int32)
    rc = torch.from_numpy(counts).cuda()
    dy, dres = rnd(T, H), rnd(T, H)

    # the tokens are taken as they arrive: row i of the normed tokens is row i of ataOut
    xd, rd, gd = x.cuda(), res.cuda(), gamma.cuda()
    wd = [w.cuda() for w in (gate, up, down)]
    n = binding.a2av_rms_norm(xd, gd, rd, 1e-6, want_y=True, want_rstd=True)
    block = ffn.ExpertBlock(W, e, T, H, N, act=act)
    y, kept = block.forward(n.y, rc, *wd)
    grads = block.backward(dy.cuda(), kept, *wd)
    dx, dgamma = binding.a2av_rms_norm_backward(grads.dAtaOut, n.h, gd, n.rstd, dres.cuda())
    assert binding.a2av_gmm_read_device_status(block.gated.workspace) == (0, 0)

    idx, sizes = R.arrival_index(counts, W, e)
    leaf = [t.double().requires_grad_(True) for t in (x, gamma, gate, up, down)]
    s = leaf[0] + res.double()
    normed = s / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-6) * leaf[1]
    h = torch.cat(R.per_expert(lambda j, r: R.act(r @ leaf[2][j], act) * (r @ leaf[3][j]), sizes, normed[idx]))
    ref = torch.cat(R.per_expert(lambda j, r: r @ leaf[4][j], sizes, h))
    want = torch.autograd.grad((ref * dy.double()).sum() + (s * dres.double()).sum(), leaf)
    tol = 5 * 2.0 ** -8
    assert _norm2(y, ref.detach()) < tol
    for got, w, name in zip((dx, dgamma, grads.dGate, grads.dUp, grads.dDown), want,
                            ("x", "gamma", "gate", "up", "down")):
        assert _norm2(got, w) < tol, name


def test_serving_in_8_bits():
    W, e, T, H, N = 2, 3, 400, 1024, 512
    g = torch.Generator().manual_seed(6)
    rnd = lambda *s, std=1.0: torch.randn(*s, generator=g) * std
    x, res, gamma = rnd(T, H).bfloat16(), rnd(T, H, std=2.0).bfloat16(), (1 + 0.1 * rnd(H)).bfloat16()
    gate, up, down = rnd(e, N, H, std=H ** -0.5), rnd(e, N, H, std=H ** -0.5), rnd(e, H, N, std=N ** -0.5)
    counts = np.random.default_rng(4).multinomial(T, np.ones(W * e) / (W * e)).astype(np.int32)
    rc = torch.from_numpy(counts).cuda()
    n = binding.a2av_rms_norm(x.cuda(), gamma.cuda(), res.cuda(), qtype="e4m3fn", mode="mx")
    guq, gus = mx_quantize(torch.cat([gate, up], dim=1), "e4m3fn")
    dq, ds = mx_quantize(down, "e4m3fn")
    block = ffn.MxExpertBlock(W, e, T, H, N)
    y = block.forward(n.codes, n.scales, rc, *[t.cuda() for t in (guq, gus, dq, ds)])
    idx, sizes = R.arrival_index(counts, W, e)
    normed = R.rms_norm(x, res, gamma, 1e-6)[1][idx]
    h = R.per_expert(lambda j, r: R.act(r @ gate[j].double().t(), "silu") * (r @ up[j].double().t()), sizes, normed)
    ref = torch.cat([hj @ down[j].double().t() for j, hj in enumerate(h)])
    assert _norm2(y, ref) < 2.0 ** -2
