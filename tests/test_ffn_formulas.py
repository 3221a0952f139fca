"""The float64 references of the expert-layer operators against central differences of their own forward forms (CPU):
what the GPU tests take for the gradient is the derivative of what they take for the value."""

import pytest
import torch

import ffn_ref as R


def _directional(f, x, v, eps=1e-5):
    return (f(x + eps * v) - f(x - eps * v)) / (2 * eps)


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
def test_activation_slopes(name):
    g = torch.linspace(-12, 12, 2001, dtype=torch.float64)
    d = (R.act(g + 1e-6, name) - R.act(g - 1e-6, name)) / 2e-6
    assert float((d - R.act_slope(g, name)).abs().max()) < 1e-8
    # what the bounds assume of the slopes and of their own slopes
    assert float(R.act_slope(g, name).abs().max()) < 1.13
    assert float(((R.act_slope(g + 1e-4, name) - R.act_slope(g - 1e-4, name)) / 2e-4).abs().max()) < 1.0


def test_norm_gradient():
    t = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=t, dtype=torch.float64)
    h, gamma, dy, dh, v, vg = rnd(5, 24), rnd(24), rnd(5, 24), rnd(5, 24), rnd(5, 24), rnd(24)
    loss = lambda h_, g_: float((R.rms_norm(h_, None, g_, 1e-3)[1] * dy).sum() + (h_ * dh).sum())
    dx, dgamma = R.rms_norm_backward(dy, dh, h, gamma, R.rms_norm(h, None, gamma, 1e-3)[2])
    assert abs(_directional(lambda z: loss(z, gamma), h, v) - float((dx * v).sum())) < 1e-6
    assert abs(_directional(lambda z: loss(h, z), gamma, vg) - float((dgamma * vg).sum())) < 1e-6


@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
def test_gated_gradient(name):
    t = torch.Generator().manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=t, dtype=torch.float64)
    W, e, H1, N, counts = 2, 3, 6, 5, [2, 0, 3, 1, 0, 2]
    A = sum(counts)
    x, wg, wu, dh = rnd(A, H1), rnd(e, H1, N), rnd(e, H1, N), rnd(A, N)
    loss = lambda x_, g_, u_: float((R.gated(x_, counts, W, e, g_, u_, name)["h"] * dh).sum())
    f = R.gated(x, counts, W, e, wg, wu, name)
    (dx, _), ((dg, _), (du, _)) = R.gated_backward(f, dh, wg, wu, name, torch.bfloat16)
    assert abs(_directional(lambda z: loss(z, wg, wu), x, z1 := rnd(A, H1)) - float((dx * z1).sum())) < 1e-6
    assert abs(_directional(lambda z: loss(x, z, wu), wg, z2 := rnd(e, H1, N)) - float((dg * z2).sum())) < 1e-6
    assert abs(_directional(lambda z: loss(x, wg, z), wu, z3 := rnd(e, H1, N)) - float((du * z3).sum())) < 1e-6
    assert float(dg[1].abs().max()) == 0.0  # the expert without rows


def test_gmm_gradient():
    t = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=t, dtype=torch.float64)
    W, e, H1, N, counts = 2, 2, 6, 5, [2, 1, 0, 3]
    x, w, dy = rnd(6, H1), rnd(e, H1, N), rnd(6, N)

    def loss(x_, w_):
        idx, sizes = R.arrival_index(counts, W, e)
        return float((torch.cat(R.per_expert(lambda j, r: r @ w_[j], sizes, x_[idx])) * dy).sum())

    idx, _ = R.arrival_index(counts, W, e)
    (dx, _), ((dw, _),) = R.gmm_backward(x[idx], counts, W, e, dy, w)
    assert abs(_directional(lambda z: loss(z, w), x, z1 := rnd(6, H1)) - float((dx * z1).sum())) < 1e-6
    assert abs(_directional(lambda z: loss(x, z), w, z2 := rnd(e, H1, N)) - float((dw * z2).sum())) < 1e-6
