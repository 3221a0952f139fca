"""mx exponents of the layer norm where a block's largest value lies within a few fp32 units of a power of two, on the GPU.

One column of each block of 32 has a gamma, the others none and no beta; its gamma and beta are searched so that one row's
value n gamma + beta comes within 2^-27.5 to 2^-22 of 1 (relative), from either side.  Every other row has a mean larger than
its deviation, about which the kernel takes its values.  Rows are sums of a multiple of 1/16 and one of 1/256: 12 bits, whose
fp32 sums are exact, and so are the squares' of a thread's 8 to 64 values (to 2^-30 of them; the mean to 12 bits leaves the
differences from it as short).  What is left are the roundings of the statistics and of y, whose errors the kernel carries
along in fp32, 2^-46 of the value.  Blocks nearer than 2^-28 to a power of two are left out."""

import numpy as np
import pytest
import torch

import ffn_ref as R
import layer_norm_ref as L
from token_permute_grouped_gb300 import binding, build

pytestmark = pytest.mark.gpu

EPS = float(np.float32(1e-5))


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()


def near(v):
    """Distance of |v| from the nearest power of two, relative."""
    m, _ = np.frexp(np.abs(v))
    return np.minimum(np.abs(2 * m - 1), np.abs(1 - m))


def rounded(v, dtype):
    return torch.from_numpy(v).to(dtype).double().numpy()


def operands(seed, rows, H, dtype):
    rng = np.random.default_rng([seed, 21])
    x = rng.integers(-64, 65, (rows, H)) / 16.0
    x[1::2] = (x[1::2] + 12.0) / 2.0  # (a mean of 6 and a deviation of about 1.2)
    x = np.round(x * 16.0) / 16.0
    res = rng.integers(-15, 16, (rows, H)) / 256.0
    s = x + res
    d = s - s.mean(1, keepdims=True)
    n = d / np.sqrt((d * d).mean(1, keepdims=True) + EPS)
    gamma, beta = np.zeros(H), np.zeros(H)
    step = 2.0 ** (-7 if dtype == torch.bfloat16 else -10)
    for b in range(H // 32):
        c = 32 * b + 7 * b % 32
        r = rng.permutation(rows)[:64]
        v = n[r, c]
        r, v = r[np.abs(v) > 0.2], v[np.abs(v) > 0.2]
        target = rng.choice([-1.0, 1.0])
        g = rounded(target / v[:, None] * (1.0 + step * np.arange(-6, 7)), dtype)
        want = target - v[:, None] * g
        be = np.stack([rounded(want * (1.0 + step * k), dtype) for k in (-1, 0, 1)], 2)
        off = np.abs((v[:, None] * g)[..., None] + be - target)
        off[off < 2.0 ** -27.5] = 1.0
        i, j, k = np.unravel_index(off.argmin(), off.shape)
        gamma[c], beta[c] = g[i, j], be[i, j, k]
    return [torch.from_numpy(a).to(dtype) for a in (x, res, gamma, beta)]


def fp32_exponents(x, res, gamma, beta):
    """The formula in plain fp32."""
    s = x.float() + res.float()
    d = s - s.mean(1, keepdim=True)
    y = d * torch.rsqrt((d * d).mean(1, keepdim=True) + EPS) * gamma.float() + beta.float()
    return torch.frexp(y.abs().unflatten(1, (-1, 32)).amax(2))[1].long() - 1


@pytest.mark.parametrize("qtype", ["e4m3fn", "e5m2"])
@pytest.mark.parametrize("rows,H,repeat,dt", [(64, 1024, 1, "bf16"), (64, 1024, 40, "bf16"), (64, 4096, 1, "fp16"), (64, 4096, 12, "fp16"),
                                              (64, 16512, 1, "bf16"), (48, 34304, 1, "fp16")])
def test_exponents_within_a_few_units_of_a_power_of_two(rows, H, repeat, dt, qtype):
    dtype = {"bf16": torch.bfloat16, "fp16": torch.float16}[dt]
    blocks, plain_wrong = {0: 0, 1: 0}, {0: 0, 1: 0}
    for seed in range(max(1, 8192 // H)):
        x, res, gamma, beta = operands(seed, rows, H, dtype)
        y = L.layer_norm(x, res, gamma, beta, EPS)["y"]
        amax = y.abs().unflatten(1, (-1, 32)).amax(2)
        want = torch.floor(torch.log2(amax)).long()
        off = torch.from_numpy(near(amax.numpy()))
        sure = off > 2.0 ** -28
        close = sure & (off < 2.0 ** -22)
        wrong = fp32_exponents(x, res, gamma, beta) != want
        for odd in (0, 1):
            blocks[odd] += int(close[odd::2].sum())
            plain_wrong[odd] += int((wrong & close)[odd::2].sum())
        r = binding.a2av_layer_norm(x.cuda().repeat(repeat, 1), gamma.cuda(), beta.cuda(), res.cuda().repeat(repeat, 1), EPS, qtype,
                                    "mx")
        got = r.scales.cpu().long().unflatten(0, (repeat, rows)) - 127 + R.F8[qtype][1]
        bad = ((got != want) & sure).any(0)
        assert not bad.any(), (int(bad.sum()), int((bad & close)[0::2].sum()), int((bad & close)[1::2].sum()), off[bad][:4].tolist())
    # rows of both kinds have such blocks, and plain fp32 puts some of each on the wrong side
    assert min(blocks.values()) > 40 and min(plain_wrong.values()) > 4, (blocks, plain_wrong)


@pytest.mark.parametrize("M", [0, 1, 3, 40, 300, 700, 1000, 1900])
@pytest.mark.parametrize("spread", [1, 4, 30])
def test_statistics_of_rows_at_any_distance_from_zero(M, spread):
    """Whole numbers around M: values, sums and the mean of a power of two of them are exact in fp32.  A thread's sum of up to
    16 squares is rounded 17 times, half a unit of fp32 each: 2^-20 of the variance, 2^-21 of rstd.  The same rows in
    several calls, one with a value that differs in a thousand."""
    rng = np.random.default_rng([M, spread])
    x = M + rng.integers(-spread, spread + 1, (40, 2048)).astype(np.float64)
    x[20:] = M
    x[20:, 77] = M + spread
    want, s = torch.from_numpy(x), torch.from_numpy(x).half()
    gamma = torch.ones(2048, dtype=torch.float16, device="cuda")
    f = L.layer_norm(s, None, gamma.cpu(), None, EPS)
    assert torch.equal(f["s"], want)
    for qtype, mode in ((None, "mx"), ("e4m3fn", "mx"), ("e4m3fn", "group128")):
        for repeat in (1, 40):
            r = binding.a2av_layer_norm(s.cuda().repeat(repeat, 1), gamma, None, None, EPS, qtype, mode, want_y=True, want_stats=True)
            mean, rstd = (t.cpu().double().view(repeat, 40) for t in (r.mean, r.rstd))
            assert bool(((mean - f["mean"]).abs() <= 2.0 ** -24 * f["mean"].abs()).all())
            assert bool(((rstd - f["rstd"]).abs() <= 2.0 ** -20 * f["rstd"]).all())
            y = r.y.cpu().double().view(repeat, 40, 2048)
            err = 2.0 ** -20 * f["y"].abs() + 2.0 ** -22
            assert bool(((y - f["y"]).abs() <= err * (1 + 2.0 ** -11) + 2.0 ** -11 * f["y"].abs() + 2.0 ** -24).all())
