"""The exponent of an mx scale for blocks whose largest magnitude lies within a few fp32 units of a power of two: it is the
one of the float64 value, on either side (on the GPU).  The inputs are searched for on the CPU."""

import numpy as np
import pytest
import torch

import ffn_ref as R
from token_permute_grouped_gb300 import binding, build

pytestmark = pytest.mark.gpu

# fp32 units (2^-24, of a value just below the power of two) that the activation's fp32 value may be off: the exponential's
# argument carries at most 5.2 units times |z| < 88 (the roundings of z's parts, of its product with log2(e) and of that
# constant), the other steps nine.
UNITS = 512
# The norm's mean is a sum of fp32 sums of 8 products: 0.3 sqrt(8) units a thread, which 512 threads average to 0.04 and the
# root halves.  Blocks within six deviations of a power of two may go either way.
EITHER = 2.0 ** -27


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()


def off_power(v):
    """v's distance from the nearest power of two, relative, and floor(log2(v)), v > 0 in float64."""
    m, ex = np.frexp(v)  # v = m 2^ex, m in [0.5, 1)
    return np.minimum(np.abs(2.0 * m - 1.0), np.abs(1.0 - m)), ex - 1


def scale_codes(v, qtype):
    return torch.from_numpy(np.clip(off_power(v)[1] - R.F8[qtype][1], -127, 127) + 127).to(torch.uint8)


@pytest.mark.parametrize("qtype", ["e4m3fn", "e5m2"])
@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
def test_gated_activation(name, qtype):
    # Every fp16 gate with a value in fp32's range (below |g| of 1/8 no rounding grows) and every fp16 mantissa of up; the
    # bf16 ones are among them.
    lo, hi = (-87.0, 87.0) if name == "silu" else (-9.2, 9.2)
    g16 = np.arange(2 ** 16, dtype=np.uint16).view(np.float16)
    g16 = g16[np.isfinite(g16) & (np.abs(g16) > 2.0 ** -3) & (g16 > lo) & (g16 < hi)]
    u16 = (np.arange(1024) + 1024).astype(np.float64) / 1024.0
    a = R.act(torch.from_numpy(g16.astype(np.float64)), name).abs().numpy()
    near_g, near_u = [], []
    for at in range(0, len(a), 512):
        off, _ = off_power(a[at:at + 512, None] * u16)
        i, j = np.nonzero(off < UNITS * 2.0 ** -24)
        near_g.append(g16[at:at + 512][i])
        near_u.append(u16[j])
    gate, up = np.concatenate(near_g), np.concatenate(near_u).astype(np.float16)
    assert (gate < -2).sum() > 8 and (gate > -2).sum() > 8
    n = len(gate)
    rows = torch.zeros(n, 2, 32, dtype=torch.float16)  # a block each: the value, among smaller ones
    rows[:, 0], rows[:, 1] = 0.5, 2.0 ** -14
    at = torch.arange(n) % 32
    rows[torch.arange(n), 0, at] = torch.from_numpy(gate)
    rows[torch.arange(n), 1, at] = torch.from_numpy(up) * torch.where(torch.arange(n) % 3 == 0, -1.0, 1.0).half()
    v = R.act(rows[:, 0].double(), name) * rows[:, 1].double()
    r = binding.a2av_glu_quant(rows.view(n, 64).cuda(), name, qtype, "mx")
    got = r.scales.cpu().view(-1)
    want = scale_codes(v.abs().amax(1).numpy(), qtype)
    wrong = torch.nonzero(got != want).view(-1)
    assert len(wrong) == 0, (len(wrong), n, gate[wrong[:8].numpy()], up[wrong[:8].numpy()])
    R.assert_codes(r.codes, r.scales, v, R.CHAIN, qtype, "mx", "codes")


@pytest.mark.parametrize("residual", [False, True])
def test_norm(residual):
    H, near = 8192, 0
    mantissas = ((torch.arange(1024) + 1024) / 1024.0).double()
    for seed in range(250):
        g = torch.Generator().manual_seed(seed)
        x = (torch.randn(1, H, generator=g)).half()
        res = (torch.randn(1, H, generator=g) * 3).half() if residual else None
        s = x.double() + (res.double() if residual else 0.0)
        n = s / torch.sqrt(s.square().mean(1, keepdim=True) + 1e-6)
        # gamma of each block's largest value: the mantissa that brings it nearest to a power of two
        top, at = n.abs().view(-1, 32).max(1)
        off, _ = off_power((top[:, None] * mantissas).numpy())
        gamma = torch.full((H // 32, 32), 2.0 ** -8, dtype=torch.float16)
        gamma[torch.arange(H // 32), at] = mantissas[torch.from_numpy(off.argmin(1))].half()
        gamma = gamma.view(H)
        amax = (n * gamma.double()).abs().view(-1, 32).amax(1).numpy()
        near += int((off_power(amax)[0] < 8 * 2.0 ** -24).sum())
        r = binding.a2av_rms_norm(x.cuda(), gamma.cuda(), None if res is None else res.cuda(), 1e-6, "e4m3fn", "mx")
        wrong = (r.scales.cpu().view(-1) != scale_codes(amax, "e4m3fn")).numpy() & (off_power(amax)[0] > EITHER)
        assert not wrong.any(), (seed, amax[wrong])
    assert near > 10  # blocks that the fp32 value alone could not decide
