"""The expert-layer operators with as many rows as they take, 2^31 - 1, of 8 values each: every row against the same
operator's result on a block of rows that the input repeats, and that block against float64 (on the GPU).  Bounds:
tests/ffn_ref.py."""

import pytest
import torch

import ffn_ref as R
from token_permute_grouped_gb300 import binding, build

pytestmark = pytest.mark.gpu

ROWS, H = 2 ** 31 - 1, 8
BLOCK = 2 ** 20
DEV = "cuda:0"


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()
    yield
    torch.cuda.empty_cache()


def rnd(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).bfloat16()


def repeated(block, dtype=torch.bfloat16):
    """ROWS rows: the block again and again, the last one short of a row."""
    out = torch.empty(ROWS, *block.shape[1:], dtype=dtype, device=DEV)
    for at in range(0, ROWS, BLOCK):
        out[at:at + BLOCK] = block[:min(BLOCK, ROWS - at)]
    return out


def assert_repeats(got, block):
    same = torch.ones((), dtype=torch.bool, device=DEV)
    for at in range(0, ROWS, BLOCK):
        same &= (got[at:at + BLOCK] == block[:min(BLOCK, ROWS - at)]).all()
    assert bool(same)


def test_norm_and_its_gradient():
    block, gamma = rnd(1, BLOCK, H).to(DEV), rnd(2, H).to(DEV)
    one = binding.a2av_rms_norm(block, gamma, None, 1e-6, want_rstd=True)
    _, y, rstd = R.rms_norm(block[:4096].cpu(), None, gamma.cpu(), 1e-6)
    R.assert_rounded(one.y[:4096], y, y.abs() * R.CHAIN, "y")
    x = repeated(block)
    r = binding.a2av_rms_norm(x, gamma, None, 1e-6, want_rstd=True)
    assert_repeats(r.y, one.y)
    assert_repeats(r.rstd, one.rstd)
    dx1, _ = binding.a2av_rms_norm_backward(one.y, block, gamma, one.rstd)
    dx, dgamma = binding.a2av_rms_norm_backward(r.y, x, gamma, r.rstd)
    assert_repeats(dx, dx1)
    terms = one.y.double() * block.double() * one.rstd.double()[:, None]
    times, rest = ROWS // BLOCK, ROWS % BLOCK
    total = lambda t: times * t.sum(0) + t[:rest].sum(0)
    # a thread adds about ROWS / (152 blocks x 8 rows) terms in a row
    lim = (ROWS / 1216 + 200) * 2.0 ** -24 * total(terms.abs())
    assert bool(((dgamma.double() - total(terms)).abs() <= lim).all())
