"""The layer norm on both sides of the rule between one vector of 8 values a thread (all rows on the SMs at once) and two, in
every band of widths, on the GPU against float64.  Bounds: tests/layer_norm_ref.py."""

import pytest
import torch

import layer_norm_ref as L
from test_gpu_layer_norm import _lib, check, dev, rnd  # noqa: F401
from token_permute_grouped_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("qtype,mode", [(None, "mx"), ("e5m2", "mx"), ("e4m3fn", "group128")])
@pytest.mark.parametrize("H", [128, 1024, 2560, 2816, 4096, 4352, 5376, 7936, 8192])
@pytest.mark.parametrize("past", [0, 1, 53])
def test_rows_that_just_fit_and_that_do_not(H, past, qtype, mode):
    threads = (H // 8 + 31) // 32 * 32
    rows = torch.cuda.get_device_properties(0).multi_processor_count * (1024 // threads) + past
    x, res = rnd(41, rows, H, mean=0.5), rnd(42, rows, H, std=2.0)
    gamma, beta = rnd(43, H, mean=1.0, std=0.2), rnd(44, H, std=0.3)
    r = binding.a2av_layer_norm(dev(x), dev(gamma), dev(beta), dev(res), 1e-5, qtype, mode, want_y=True, want_stats=True)
    check(L.layer_norm(x, res, gamma, beta, 1e-5), r, qtype, mode)
