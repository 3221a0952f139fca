"""Argument checks of the layer norm's C ABI and binding, and its float64 gradient against differences (no GPU needed:
every call returns before the library touches CUDA)."""

import ctypes

import pytest
import torch

import layer_norm_ref as L
from token_permute_grouped_gb300 import binding, build

NAMES = binding.STATUS_NAMES
OK, NULLPTR, INVALID, UNSUPPORTED, WORKSPACE = ("A2AV_OK", "A2AV_ERR_NULLPTR", "A2AV_ERR_INVALID",
                                                "A2AV_ERR_UNSUPPORTED", "A2AV_ERR_WORKSPACE")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def ptr(i):
    return 0x100000 + 0x10000 * i


def norm(lib, desc=None, **kw):
    d = dict(rows=4, H=256, x_stride=256, residual_stride=256, dtype=0, qtype=0, qmode=0, eps=1e-5)
    d.update(desc or {})
    names = ["x", "residual", "gamma", "beta", "h", "y", "codes", "scales", "mean", "rstd"]
    args = [kw.get(n, ptr(i)) for i, n in enumerate(names)]
    return NAMES[lib.a2av_layer_norm(ctypes.byref(binding.LayerNormDesc(**d)), *args, None)]


@pytest.mark.parametrize("desc,kw,want", [
    ({"rows": -1}, {}, INVALID), ({"rows": 2 ** 31}, {}, INVALID), ({"H": 0}, {}, INVALID), ({"H": 65536}, {}, INVALID),
    ({"dtype": 2}, {}, INVALID), ({"eps": -1.0}, {}, INVALID), ({"eps": float("nan")}, {}, INVALID),
    ({"x_stride": 248}, {}, INVALID), ({"residual_stride": 8}, {}, INVALID), ({"x_stride": 260}, {}, UNSUPPORTED),
    ({"qtype": 3}, {}, INVALID), ({"qtype": 2}, {}, INVALID), ({"qmode": 2}, {}, INVALID),
    ({"H": 264, "x_stride": 264, "residual_stride": 264}, {}, INVALID),
    ({}, {"x": 0}, NULLPTR), ({}, {"gamma": 0}, NULLPTR), ({}, {"codes": 0}, NULLPTR), ({}, {"scales": 0}, NULLPTR),
    ({"qtype": -1}, {}, INVALID),
    ({"qtype": -1}, {"codes": 0, "scales": 0, "h": 0, "y": 0, "mean": 0, "rstd": 0}, NULLPTR),
    ({}, {"x": ptr(0) + 8}, UNSUPPORTED), ({}, {"beta": ptr(0) + 2}, UNSUPPORTED), ({}, {"codes": ptr(0) + 4}, UNSUPPORTED),
    ({}, {"mean": ptr(0) + 2}, UNSUPPORTED), ({}, {"rstd": ptr(0) + 2}, UNSUPPORTED),
    ({"rows": 0}, {"x": 0, "residual": 0, "beta": 0, "h": 0, "y": 0, "codes": 0, "scales": 0, "mean": 0, "rstd": 0}, OK),
])
def test_checks(lib, desc, kw, want):
    assert norm(lib, desc, **kw) == want


def test_null_descriptor(lib):
    assert NAMES[lib.a2av_layer_norm(None, *[ptr(i) for i in range(10)], None)] == NULLPTR


def backward(lib, rows=400, H=256, dtype=0, wsbytes=1 << 20, **kw):
    names = ["dy", "dh", "h", "gamma", "mean", "rstd", "dx", "dgamma", "dbeta", "workspace"]
    args = [kw.get(n, ptr(i)) for i, n in enumerate(names)]
    return NAMES[lib.a2av_layer_norm_backward(rows, H, dtype, *args, wsbytes, None)]


@pytest.mark.parametrize("kw,want", [
    ({"rows": -1}, INVALID), ({"H": 0}, INVALID), ({"H": 65536}, INVALID), ({"dtype": 2}, INVALID),
    ({"H": 12}, UNSUPPORTED), ({"dy": 0}, NULLPTR), ({"h": 0}, NULLPTR), ({"gamma": 0}, NULLPTR), ({"mean": 0}, NULLPTR),
    ({"rstd": 0}, NULLPTR), ({"dx": 0}, NULLPTR), ({"dgamma": 0}, NULLPTR), ({"dbeta": 0}, NULLPTR),
    ({"workspace": 0}, NULLPTR), ({"wsbytes": 16}, WORKSPACE), ({"workspace": ptr(9) + 16}, WORKSPACE),
    ({"dh": ptr(1) + 8}, UNSUPPORTED), ({"dbeta": ptr(1) + 4}, UNSUPPORTED), ({"mean": ptr(1) + 2}, UNSUPPORTED),
    ({"rows": 0, "dgamma": 0, "dbeta": 0}, OK),
])
def test_backward_checks(lib, kw, want):
    assert backward(lib, **kw) == want


def test_binding_refuses_what_is_not_on_a_gpu():
    x, gamma = torch.zeros(4, 256, dtype=torch.bfloat16), torch.ones(256, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="CUDA"):
        binding.a2av_layer_norm(x, gamma)
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        binding.a2av_layer_norm(x.float(), gamma)
    with pytest.raises(TypeError, match="CUDA"):
        binding.a2av_layer_norm_backward(x, x, gamma, torch.zeros(4), torch.zeros(4))


def test_gradient_is_the_derivative():
    t = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=t, dtype=torch.float64)
    h, gamma, beta, dy, dh = rnd(5, 24) + 2.0, rnd(24), rnd(24), rnd(5, 24), rnd(5, 24)
    loss = lambda h_, g_, b_: float((L.layer_norm(h_, None, g_, b_, 1e-3)["y"] * dy).sum() + (h_ * dh).sum())
    f = L.layer_norm(h, None, gamma, beta, 1e-3)
    grads = L.layer_norm_backward(dy, dh, h, gamma, f["mean"], f["rstd"])
    at = [h, gamma, beta]
    for i, g in enumerate(grads):
        v = rnd(*at[i].shape)
        up, down = [list(at) for _ in range(2)]
        up[i], down[i] = at[i] + 1e-5 * v, at[i] - 1e-5 * v
        assert abs((loss(*up) - loss(*down)) / 2e-5 - float((g * v).sum())) < 1e-6
