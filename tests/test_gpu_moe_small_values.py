"""Gated values of any size between the two products of the expert layer for a few tokens, on the GPU against float64.

A token is 1 or less in one place and 0 elsewhere, so that its gate and up products are single, exact products: what is left
between the block's values and y is the activation (CHAIN, tests/ffn_ref.py), the two summands of the element type, and the
second product.  bf16: two summands hold a value to 2 u^2 = 2^-15 of it.  fp16: the first holds half the value to 2^-11 of
it, the second 1024 times the rest to 2^-11 of that, or to half of fp16's step: 2^-22 of the value, or 2^-25 / 1024."""

import pytest
import torch

import ffn_ref as R
from token_permute_grouped_gb300 import binding, build

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()


def inputs(seed, sizes, E, H, N, dtype):
    """Token t is sizes[t] in place t; router, gate and up of the places' own."""
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)
    T = len(sizes)
    x = torch.zeros(T, H)
    x[torch.arange(T), torch.arange(T)] = torch.tensor(sizes)
    # (values around 1, of both signs: none is much smaller than the others)
    near_one = lambda *s: (0.5 + torch.rand(*s, generator=g)) * torch.sign(rnd(*s))
    return {"x": x.to(dtype), "router": rnd(E, H).to(dtype), "gate": near_one(E, H, N).to(dtype),
            "up": near_one(E, H, N).to(dtype), "down": near_one(E, N, H).to(dtype)}


def run(s, K, scale, dtype):
    T, H = s["x"].shape
    E, _, N = s["gate"].shape
    plan = binding.MoePlan(T, E, K, H, N, dtype, scale=scale)
    r = plan.run(*[s[k].cuda() for k in ("x", "router", "gate", "up", "down")])
    assert binding.a2av_gmm_read_device_status(plan.workspace) == (0, 0)
    return r


def values(s, t, e):
    """The block's values of token t at expert e."""
    g, u = s["x"][t].double() @ s["gate"][e].double(), s["x"][t].double() @ s["up"][e].double()
    return R.act(g, "silu") * u


def check(s, r, dtype):
    T, K = r.experts.shape
    N = s["gate"].shape[2]
    y = torch.zeros(s["x"].shape, dtype=torch.float64)
    err = torch.zeros_like(y)
    for t in range(T):
        for k in range(K):
            e, w = int(r.experts[t, k]), float(r.weights[t, k])
            h, wd = values(s, t, e), s["down"][e].double()
            held = 2.0 ** -15 * h.abs() if dtype == torch.bfloat16 else 2.0 ** -22 * h.abs() + 2.0 ** -35
            eh = R.CHAIN * h.abs() + held
            d = w * (h @ wd)
            y[t] += d
            err[t] += abs(w) * (eh @ wd.abs() + (2 * N + 8) * 2.0 ** -23 * ((h.abs() + eh) @ wd.abs()))
            err[t] += (K + 2) * 2.0 ** -23 * (d.abs() + y[t].abs())
    # (fp16 ends at 65504: from half a step above it, 65520, the nearest value is an infinity.  It has to be one where all
    # values within err lie there, and may be one where some do.)
    inf = torch.sign(y) * float("inf")
    far = torch.tensor(dtype == torch.float16)
    must, may = far & (y.abs() - err >= 65520.0), far & (y.abs() + err >= 65520.0)
    R.assert_rounded(r.y, torch.where(must | may & (r.y.cpu().double() == inf), inf, y), err, "y")


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
@pytest.mark.parametrize("T,E,K,H,N", [(7, 3, 2, 64, 136), (20, 2, 2, 72, 520), (64, 2, 2, 64, 72), (61, 40, 3, 136, 328)])
def test_small_values(T, E, K, H, N, dt):
    # Values of about a quarter of the sizes' squares: 1e-3 to 1e-9, and weights that bring y into fp16's middle.
    sizes = [(4 * 10.0 ** -(3 + t % 7)) ** 0.5 for t in range(T)]
    s = inputs(1, sizes, E, H, N, DT[dt])
    check(s, run(s, K, 2.0 ** 20, DT[dt]), DT[dt])


def test_values_up_to_twice_the_range_of_fp16():
    s = inputs(2, [1.0, 1.0, 1.0], 1, 64, 72, torch.float16)
    g = torch.Generator().manual_seed(3)
    s["gate"][:] = 300.0
    s["up"] = ((230.0 + 200.0 * torch.rand(1, 64, 72, generator=g)) * torch.sign(torch.randn(1, 64, 72, generator=g))).half()
    s["down"] = (s["down"].float() * 1e-3).half()
    v = values(s, 0, 0).abs()
    assert float(v.max()) > 120000 and float(v.max()) < 131008 and float(v.min()) > 65504
    check(s, run(s, 1, 1.0, torch.float16), torch.float16)


@pytest.mark.parametrize("dt", ["fp16", "bf16"])
def test_an_infinite_weight_meets_values_of_any_size(dt):
    """An infinity times a value that is not 0 is an infinity of their signs; times 0 it is a NaN."""
    sizes = [2.0 * 10.0 ** -(i / 2) for i in range(9)] + [0.0]
    s = inputs(4, sizes, 1, 64, 72, DT[dt])
    s["down"][0, 5, 7] = float("inf")
    s["down"][0, 70, 8] = float("-inf")
    y = run(s, 1, 1.0, DT[dt]).y.cpu().double()
    for t in range(len(sizes)):
        h = values(s, t, 0)
        want = torch.stack((h[5], -h[70])) * float("inf")
        assert torch.equal(y[t, 7:9], want) if t < 9 else bool(torch.isnan(y[t, 7:9]).all())
    rest = torch.ones(64, dtype=torch.bool)
    rest[7:9] = False
    assert bool(torch.isfinite(y[:, rest]).all())
