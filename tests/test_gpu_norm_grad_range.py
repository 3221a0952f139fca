"""The norm's gradient for rows of very small and very large values, whose squared reciprocal root is out of fp32's range,
against float64 (on the GPU).  Bounds: tests/ffn_ref.py."""

import pytest
import torch

import ffn_ref as R
from token_permute_grouped_gb300 import binding, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()


@pytest.mark.parametrize("H", [128, 2048, 20000, 40000])
@pytest.mark.parametrize("rows", [3, 600])
def test_scales_of_rows(rows, H):
    g = torch.Generator().manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=g)
    scale = torch.tensor([1e-25, 1e25, 1e-18, 1e18, 1e-30, 1e30, 1.0]).repeat(rows)[:rows, None]
    h = (rnd(rows, H) * scale).bfloat16()
    dy, gamma = (rnd(rows, H) * 0.1).bfloat16(), (rnd(H) * 0.2 + 1.0).bfloat16()
    rstd = (1.0 / h.double().square().mean(1).sqrt()).float()
    dx, dgamma = binding.a2av_rms_norm_backward(dy.cuda(), h.cuda(), gamma.cuda(), rstd.cuda())
    rx, rg = R.rms_norm_backward(dy, None, h, gamma, rstd)
    n, a = h.double() * rstd.double()[:, None], dy.double() * gamma.double()
    err = R.CHAIN * rstd.double()[:, None] * (a.abs() + n.abs() * (a * n).abs().mean(1, keepdim=True)) + 2.0 ** -23 * rx.abs()
    R.assert_rounded(dx, rx, err, "dx")
    lim = (dy.double() * n).abs().sum(0) * (rows + 64) * 2.0 ** -24 + 1e-30
    assert bool(((dgamma.cpu().double() - rg).abs() <= lim).all())
