"""The norm's gradient over few rows, taken by one block or by several, at both sides of each limit (needs a GB300).
Against float64; bounds as in test_gpu_ffn.py."""

import pytest
import torch

import ffn_ref as R
from token_permute_grouped_gb300 import binding, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()


@pytest.mark.parametrize("H", [8, 136, 560, 2048, 4096, 8192, 8200])
@pytest.mark.parametrize("rows", [1, 2, 3, 4, 5, 8, 9, 16, 17, 31, 32, 33, 64, 65, 127, 128, 129, 255, 256, 257])
def test_few_rows(rows, H):
    g = torch.Generator().manual_seed(rows * 10007 + H)
    rnd = lambda *s, std=1.0, mean=0.0: (torch.randn(*s, generator=g) * std + mean).bfloat16()
    h, dy, gamma = rnd(rows, H, std=2.0), rnd(rows, H, std=0.1), rnd(H, std=0.2, mean=1.0)
    dh = rnd(rows, H, std=0.1) if rows % 2 else None
    rstd = R.rms_norm(h, None, gamma, 1e-6)[2].float()
    args = [None if t is None else t.cuda() for t in (dy, h, gamma, rstd, dh)]
    guard = torch.full((H + 64,), 5.0, device="cuda")
    dx, dgamma = binding.a2av_rms_norm_backward(*args, dgamma=guard[:H])
    rx, rg = R.rms_norm_backward(dy, dh, h, gamma, rstd)
    n = h.double() * rstd.double()[:, None]
    a = dy.double() * gamma.double()
    err = R.CHAIN * rstd.double()[:, None] * (a.abs() + n.abs() * (a * n).abs().mean(1, keepdim=True)) + 2.0 ** -23 * rx.abs()
    R.assert_rounded(dx, rx, err, "dx")
    lim = (dy.double() * n).abs().sum(0) * (rows + 64) * 2.0 ** -24 + 1e-30
    assert bool(((dgamma.cpu().double() - rg).abs() <= lim).all())
    assert bool((guard[H:] == 5.0).all())
    again = binding.a2av_rms_norm_backward(*args)
    assert torch.equal(again[0].view(torch.int16), dx.view(torch.int16)) and torch.equal(again[1], dgamma)
