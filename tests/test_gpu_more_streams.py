"""The layer norm, the product with a scale per 128 and the few-token expert layer with as many rows as a norm takes, and on
streams: what a call makes for itself belongs to the stream that works on it (needs a GB300)."""

import pytest
import torch

import layer_norm_ref as L
import ffn_ref as R
from token_permute_grouped_gb300 import binding, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    yield
    torch.cuda.empty_cache()


def rnd(*shape):
    return torch.randn(*shape, device="cuda").bfloat16()


def calls():
    rows, H, e, N = 400, 1024, 2, 256
    x, dy, gamma, beta = rnd(rows, H), rnd(rows, H), rnd(H), rnd(H)
    f = binding.a2av_layer_norm(x, gamma, beta, want_stats=True)
    rc = torch.tensor([100, 100, 100, 100], dtype=torch.int32, device="cuda")
    codes = lambda *s: torch.randint(0, 120, s, dtype=torch.uint8, device="cuda")
    q, sc, w, ws = codes(rows, H), torch.rand(rows, H // 128, device="cuda"), codes(e, N, H), torch.rand(e, 2, H // 128, device="cuda")
    g128 = binding.G128Plan(2, e, rows, H, N)
    moe = binding.MoePlan(4, 8, 2, H, N)
    x4, router, gate, up, down = rnd(4, H), rnd(8, H), rnd(8, H, N), rnd(8, H, N), rnd(8, N, H)
    return {
        "norm": lambda s: binding.a2av_layer_norm(x, gamma, beta, dy, 1e-5, "e4m3fn", "mx", True, True, stream=s),
        "norm_backward": lambda s: binding.a2av_layer_norm_backward(dy, x, gamma, f.mean, f.rstd, stream=s),
        "g128": lambda s: (g128.run(q, sc, rc, w, ws, stream=s),),
        "moe": lambda s: moe.run(x4, router, gate, up, down, stream=s),
    }


@pytest.mark.parametrize("name", ["norm", "norm_backward", "g128", "moe"])
def test_outputs_are_of_the_stream_that_writes_them(name):
    call = calls()[name]
    first = [t for t in call(None) if t is not None]
    sizes = [t.numel() * t.element_size() for t in first]
    torch.cuda.synchronize()
    blocks = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in sizes]  # used by the current stream, and given back
    mine = {b.data_ptr() for b in blocks}
    del blocks
    got = [t for t in call(torch.cuda.Stream()) if t is not None]
    torch.cuda.synchronize()
    assert not mine & {t.data_ptr() for t in got}
    for a, b in zip(first, got):
        assert torch.equal(a, b)


def test_norm_and_its_gradient_of_the_most_rows():
    """2^31 - 1 rows of 8 values: every row against the same operator's result on a block of rows that the input repeats,
    and that block against float64."""
    ROWS, H, BLOCK = 2 ** 31 - 1, 8, 2 ** 20
    g = torch.Generator(device="cuda").manual_seed(1)
    block, gamma, beta = (torch.randn(*s, generator=g, device="cuda").bfloat16() for s in ((BLOCK, H), (H,), (H,)))
    one = binding.a2av_layer_norm(block, gamma, beta, want_stats=True)
    f = L.layer_norm(block[:4096].cpu(), None, gamma.cpu(), beta.cpu(), 1e-5)
    R.assert_rounded(one.y[:4096], f["y"], f["ey"], "y")

    def same(got, want):
        ok = torch.ones((), dtype=torch.bool, device="cuda")
        for at in range(0, ROWS, BLOCK):
            ok &= (got[at:at + BLOCK] == want[:min(BLOCK, ROWS - at)]).all()
        return bool(ok)

    x = torch.empty(ROWS, H, dtype=torch.bfloat16, device="cuda")
    for at in range(0, ROWS, BLOCK):
        x[at:at + BLOCK] = block[:min(BLOCK, ROWS - at)]
    r = binding.a2av_layer_norm(x, gamma, beta, want_stats=True)
    assert same(r.y, one.y) and same(r.mean, one.mean) and same(r.rstd, one.rstd)
    dx1, _, _ = binding.a2av_layer_norm_backward(one.y, block, gamma, one.mean, one.rstd)
    dx, dgamma, dbeta = binding.a2av_layer_norm_backward(r.y, x, gamma, r.mean, r.rstd)
    assert same(dx, dx1)
    dy = one.y.double()
    n = (block.double() - one.mean.double()[:, None]) * one.rstd.double()[:, None]
    total = lambda t: ROWS // BLOCK * t.sum(0) + t[:ROWS % BLOCK].sum(0)
    for got, terms in ((dgamma, dy * n), (dbeta, dy)):
        # a thread adds about ROWS / (152 blocks x 8 rows) terms in a row
        lim = (ROWS / 1216 + 200) * 2.0 ** -24 * total(terms.abs())
        assert bool(((got.double() - total(terms)).abs() <= lim).all())
