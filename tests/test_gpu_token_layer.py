"""Layers put together from the norms, the product with a scale per 128 and the few-token expert layer
(token_permute_grouped_gb300/ffn.py), on the GPU against float64.  Errors are compared in the 2-norm; a tensor that is
rounded to bf16 on the way adds at most u = 2^-8 of its own size, an E4M3FN operand at most 2^-4 of it (three fraction bits;
the scale of a block is its largest value over 448, so none saturates)."""

import numpy as np
import pytest
import torch

import ffn_ref as R
import g128_ref as G
import layer_norm_ref as L
import moe_ref as M
from token_permute_grouped_gb300 import binding, build, ffn

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()


def norm2(got, ref):
    return float((got.double().cpu() - ref).norm() / ref.norm())


@pytest.mark.parametrize("W,e,T,H,N,act", [(1, 4, 300, 256, 192, "silu"), (4, 3, 700, 520, 328, "gelu_tanh")])
def test_training_step_behind_a_layer_norm(W, e, T, H, N, act):
    """Tokens -> layer norm with residual -> rows of the experts -> block -> gradients of everything.  At most five roundings
    stand behind any output."""
    g = torch.Generator().manual_seed(5)
    rnd = lambda *s, std=1.0, mean=0.0: (torch.randn(*s, generator=g) * std + mean).bfloat16()
    x, res, gamma, beta = rnd(T, H), rnd(T, H, std=2.0, mean=1.0), rnd(H, std=0.1, mean=1.0), rnd(H, std=0.1)
    gate, up, down = rnd(e, H, N, std=H ** -0.5), rnd(e, H, N, std=H ** -0.5), rnd(e, N, H, std=N ** -0.5)
    counts = np.random.default_rng(3).multinomial(T, np.ones(W * e) / (W * e)).astype(np.int32)
    rc, dy, dres = torch.from_numpy(counts).cuda(), rnd(T, H), rnd(T, H)
    gd, wd = gamma.cuda(), [w.cuda() for w in (gate, up, down)]
    n = binding.a2av_layer_norm(x.cuda(), gd, beta.cuda(), res.cuda(), 1e-5, want_stats=True)
    block = ffn.ExpertBlock(W, e, T, H, N, act=act)
    y, kept = block.forward(n.y, rc, *wd)
    grads = block.backward(dy.cuda(), kept, *wd)
    dx, dgamma, dbeta = binding.a2av_layer_norm_backward(grads.dAtaOut, n.h, gd, n.mean, n.rstd, dres.cuda())

    idx, sizes = R.arrival_index(counts, W, e)
    leaf = [t.double().requires_grad_(True) for t in (x, gamma, beta, gate, up, down)]
    s = leaf[0] + res.double()
    d = s - s.mean(1, keepdim=True)
    normed = d / torch.sqrt((d * d).mean(1, keepdim=True) + 1e-5) * leaf[1] + leaf[2]
    h = torch.cat(R.per_expert(lambda j, r: R.act(r @ leaf[3][j], act) * (r @ leaf[4][j]), sizes, normed[idx]))
    ref = torch.cat(R.per_expert(lambda j, r: r @ leaf[5][j], sizes, h))
    want = torch.autograd.grad((ref * dy.double()).sum() + (s * dres.double()).sum(), leaf)
    tol = 5 * 2.0 ** -8
    assert norm2(y, ref.detach()) < tol
    for got, w in zip((dx, dgamma, dbeta, grads.dGate, grads.dUp, grads.dDown), want):
        assert norm2(got, w) < tol


@pytest.mark.parametrize("W,e,T,H,N", [(2, 3, 260, 512, 256), (4, 2, 9, 256, 128), (1, 2, 40, 1024, 384)])
def test_serving_block_with_scales_per_128(W, e, T, H, N):
    """Layer norm to codes -> block.  Against the layer in float64 with the weights' quantised values: two operands are
    quantised on the way, 2^-4 each, and two results rounded."""
    g = torch.Generator().manual_seed(6)
    x = torch.randn(T, H, generator=g).bfloat16()
    gamma, beta = (1 + 0.1 * torch.randn(H, generator=g)).bfloat16(), (0.1 * torch.randn(H, generator=g)).bfloat16()
    gu = G.quantise(torch.randn(e, 2 * N, H, generator=g) * H ** -0.5, "e4m3fn", 128)
    dn = G.quantise(torch.randn(e, H, N, generator=g) * N ** -0.5, "e4m3fn", 128)
    counts = np.random.default_rng(4).multinomial(T, np.ones(W * e) / (W * e)).astype(np.int32)
    n = binding.a2av_layer_norm(x.cuda(), gamma.cuda(), beta.cuda(), None, 1e-5, "e4m3fn", "group128")
    block = ffn.G128ExpertBlock(W, e, T, H, N)
    y = block.forward(n.codes, n.scales, torch.from_numpy(counts).cuda(), *[t.cuda() for t in (*gu, *dn)])
    assert binding.a2av_gmm_read_device_status(block.first.workspace) == (0, 0)
    assert binding.a2av_gmm_read_device_status(block.down.workspace) == (0, 0)

    idx, sizes = R.arrival_index(counts, W, e)
    normed = L.layer_norm(x, None, gamma, beta, 1e-5)["y"][idx]
    wgu, wd = G.values(*gu, "e4m3fn", 128), G.values(*dn, "e4m3fn", 128)
    g_u = torch.cat(R.per_expert(lambda j, r: r @ wgu[j].t(), sizes, normed))
    h = R.act(g_u[:, :N], "silu") * g_u[:, N:]
    ref = torch.cat(R.per_expert(lambda j, r: r @ wd[j].t(), sizes, h))
    assert norm2(y, ref) < 2 * 2.0 ** -4 + 2 * 2.0 ** -8


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("T", [1, 6, 64])
def test_decode_step(T, norm):
    """Norm with residual -> a few tokens' expert layer, twice: the second layer takes the first one's y and stream.  The
    choice and the values follow from the normed rows that the layer was given, so they are checked as such."""
    E, K, H, N = 12, 3, 512, 264
    g = torch.Generator().manual_seed(7)
    rnd = lambda *s, std=1.0, mean=0.0: (torch.randn(*s, generator=g) * std + mean).bfloat16()
    x, res, gamma, beta = rnd(T, H), rnd(T, H), rnd(H, std=0.1, mean=1.0), rnd(H, std=0.1) if norm == "layer" else None
    w = [rnd(E, H, std=1.5 * H ** -0.5), rnd(E, H, N, std=H ** -0.5), rnd(E, H, N, std=H ** -0.5), rnd(E, N, H, std=N ** -0.5)]
    layer = ffn.TokenLayer(T, E, K, H, N)
    wd, b = [t.cuda() for t in w], None if beta is None else beta.cuda()
    first = layer.forward(x.cuda(), res.cuda(), gamma.cuda(), *wd, beta=b)
    second = layer.forward(first.y, None, gamma.cuda(), *wd, beta=b)
    assert binding.a2av_gmm_read_device_status(layer.moe.workspace) == (0, 0)
    for a, r, out in ((x, res, first), (first.y.cpu(), None, second)):
        if norm == "layer":
            f = L.layer_norm(a, r, gamma, beta, 1e-6)
            s, n = f["s"], f["y"]
        else:
            s, n, _ = R.rms_norm(a, r, gamma, 1e-6)
        chosen, weights = out.experts.cpu().long(), out.weights.cpu().double()
        y, _ = M.values(n, chosen, weights, torch.zeros(T, K), *w[1:], "silu", s, torch.bfloat16)
        # the normed rows and the stream are rounded, and the result
        assert norm2(out.y, y) < 3 * 2.0 ** -8
        assert bool((weights.sum(1) - 1).abs().max() < 2.0 ** -20)
