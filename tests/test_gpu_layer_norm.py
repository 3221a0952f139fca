"""The layer norm and its gradient on the GPU against float64 (needs a GB300).  Bounds: tests/layer_norm_ref.py."""

import numpy as np
import pytest
import torch

import ffn_ref as R
import layer_norm_ref as L
from token_permute_grouped_gb300 import binding, build

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
COMBOS = [(None, "mx"), ("e4m3fn", "mx"), ("e5m2", "mx"), ("e4m3fn", "group128"), ("e5m2", "group128"),
          ("int8", "group128")]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()


def rnd(seed, *shape, dtype=torch.bfloat16, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std + mean).to(dtype)


def dev(*ts):
    out = [None if t is None else t.cuda() for t in ts]
    return out[0] if len(out) == 1 else out


def check(f, r, qtype, mode, residual=True, want_y=True):
    if residual:
        R.assert_rounded(r.h, f["s"], f["s"].abs() * 2.0 ** -24, "h")
    if want_y:
        R.assert_rounded(r.y, f["y"], f["ey"], "y")
    if qtype:
        # An error relative to a value is at most that of its block's largest, times their ratio: codes are compared
        # with the rows whose errors are everywhere small against the values' grid.
        rows = (f["ey"].amax(1) < 2.0 ** -14 * f["y"].abs().unflatten(1, (-1, 32 if mode == "mx" else 128)).amax(2).amin(1))
        rows |= ~torch.isfinite(f["y"]).all(1)
        assert bool(rows.any()) or f["y"].shape[0] == 0
        codes, scales = r.codes.cpu()[rows], r.scales.cpu()[rows]
        assert_codes(codes, scales, f["y"][rows], f["ey"][rows], qtype, mode)
    if r.mean is not None:
        ok = torch.isfinite(f["mean"])
        assert bool(((r.mean.cpu().double() - f["mean"]).abs() <= f["em"] + 2.0 ** -24 * f["mean"].abs())[ok].all())
        ok = torch.isfinite(f["rstd"])
        assert bool(((r.rstd.cpu().double() - f["rstd"]).abs() <= f["rel"] * f["rstd"])[ok].all())


def assert_codes(codes, scales, y, err, qtype, mode):
    """codes and scales stand for values within err (absolute) of y."""
    block = 32 if mode == "mx" else 128
    b, eb = y.unflatten(1, (-1, block)), err.unflatten(1, (-1, block))
    c = R.decode(codes, qtype).reshape(b.shape)
    finite = torch.isfinite(b).all(2)
    amax, e = b.abs().amax(2), eb.amax(2)
    if mode == "mx":
        emax = R.F8[qtype][1]
        sc = scales.long().reshape(amax.shape)
        assert torch.equal(sc == 255, ~finite)
        want = lambda m: (torch.floor(torch.log2(m.clamp_min(2.0 ** -140))) - emax).clamp(-127, 127).long() + 127
        assert bool(((sc >= want(amax - e)) & (sc <= want(amax + e)))[finite].all())
        scale, top = torch.exp2(sc.double() - 127), R.F8[qtype][2]
    else:
        top = R.QMAX[qtype]
        scale = scales.double().reshape(amax.shape)
        assert torch.equal(torch.isnan(scale), ~finite)
        assert bool(((scale - amax.clamp_min(2.0 ** -100) / top).abs() <= e / top + amax / top * 2.0 ** -22)[finite].all())
    v = (b / scale[..., None])
    slack = eb / scale[..., None] + v.abs() * (2.0 ** -21 + (e / amax.clamp_min(1e-300))[..., None])
    if qtype == "int8":
        half = torch.full_like(v, 0.5)
    else:
        _, _, _, mant, emin = R.F8[qtype]
        half = torch.exp2(torch.floor(torch.log2((v.abs() + slack).clamp_min(2.0 ** emin))).clamp_min(emin) - mant - 1)
    bad = ~((c - v.clamp(-top, top)).abs() <= half + slack) & finite[..., None]
    assert not bad.any(), (int(bad.sum()), torch.nonzero(bad)[:4].tolist(), c[bad][:4], v[bad][:4])


@pytest.mark.parametrize("qtype,mode", COMBOS)
@pytest.mark.parametrize("rows,H", [(1, 128), (1, 7168), (3, 256), (37, 1408), (200, 4096), (400, 2048), (5, 16512),
                                    (2, 34304), (3, 65408)])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_norm(rows, H, dt, qtype, mode):
    dtype = DT[dt]
    x, res = rnd(1, rows, H, dtype=dtype, mean=0.5), rnd(2, rows, H, dtype=dtype, std=3.0)
    gamma, beta = rnd(3, H, dtype=dtype, std=0.2, mean=1.0), rnd(4, H, dtype=dtype, std=0.3)
    r = binding.a2av_layer_norm(dev(x), dev(gamma), dev(beta), dev(res), 1e-5, qtype, mode, want_y=True, want_stats=True)
    check(L.layer_norm(x, res, gamma, beta, 1e-5), r, qtype, mode)


@pytest.mark.parametrize("H", [8, 40, 136, 1000, 8200, 65528])
@pytest.mark.parametrize("rows", [1, 7, 300])
def test_odd_widths_without_beta(H, rows):
    x, gamma = rnd(5, rows, H, dtype=torch.float16), rnd(6, H, dtype=torch.float16)
    r = binding.a2av_layer_norm(dev(x), dev(gamma), eps=1e-6, want_stats=True)
    assert r.h is None and r.codes is None
    check(L.layer_norm(x, None, gamma, None, 1e-6), r, None, "mx", residual=False)


def test_rows_far_from_zero():
    # A mean a thousand times the deviation: the squares are summed about the mean.
    x, gamma, beta = rnd(7, 40, 2048, std=1.0, mean=1000.0, dtype=torch.float16), rnd(8, 2048, dtype=torch.float16), \
        rnd(9, 2048, dtype=torch.float16)
    r = binding.a2av_layer_norm(dev(x), dev(gamma), dev(beta), eps=1e-5, want_stats=True)
    check(L.layer_norm(x, None, gamma, beta, 1e-5), r, None, "mx", residual=False)
    # equal values: nothing is left but beta
    same = torch.full((3, 1000), 3.0, dtype=torch.bfloat16, device="cuda")
    b = rnd(10, 1000)
    r = binding.a2av_layer_norm(same, torch.ones(1000, dtype=torch.bfloat16, device="cuda"), dev(b))
    assert torch.equal(r.y.cpu(), b.expand(3, 1000))


def test_only_codes_strides_broadcast_in_place_and_no_rows():
    wide, gamma, beta = rnd(11, 50, 640), rnd(12, 512, mean=1.0, std=0.1), rnd(13, 512)
    x, one = wide.cuda()[:, 64:576], rnd(14, 1, 512)
    r = binding.a2av_layer_norm(x, dev(gamma), dev(beta), dev(one).expand(50, 512), 1e-5, "e5m2", "group128",
                                want_stats=True)
    assert r.y is None
    check(L.layer_norm(wide[:, 64:576], one.expand(50, 512), gamma, beta, 1e-5), r, "e5m2", "group128", want_y=False)
    res = rnd(15, 50, 512)
    buf = dev(res)
    again = binding.a2av_layer_norm(x, dev(gamma), dev(beta), buf, 1e-5, "e5m2", "group128", want_stats=True,
                                    out=r._replace(h=buf))
    assert again.h.data_ptr() == buf.data_ptr() and again.codes.data_ptr() == r.codes.data_ptr()
    check(L.layer_norm(wide[:, 64:576], res, gamma, beta, 1e-5), again, "e5m2", "group128", want_y=False)
    none = binding.a2av_layer_norm(x[:0], dev(gamma), qtype="e4m3fn", want_y=True)
    assert none.codes.shape == (0, 512) and none.y.shape == (0, 512)
    torch.cuda.synchronize()


@pytest.mark.parametrize("qtype,mode", COMBOS[1:])
def test_zero_and_non_finite_rows(qtype, mode):
    x, gamma = rnd(16, 8, 256), torch.ones(256, dtype=torch.bfloat16)
    beta = torch.zeros(256, dtype=torch.bfloat16)
    x[1] = 0.0                          # eps alone under the root: zeros
    x[3, 17] = float("nan")
    x[5, 200] = float("inf")            # an infinite mean: every value NaN
    x[6, ::2], x[6, 1::2] = 3e38, -3e38  # finite, but its squares are not: rstd 0, every value 0
    gamma[40] = float("inf")            # one column's values infinite in every row
    beta[41] = float("nan")
    r = binding.a2av_layer_norm(dev(x), dev(gamma), dev(beta), None, 1e-5, qtype, mode, want_y=True)
    s = x.float()
    with np.errstate(all="ignore"):
        d = s - s.mean(1, keepdim=True)
        y = (d * torch.rsqrt((d * d).mean(1, keepdim=True) + 1e-5) * gamma.float() + beta.float()).double()
    err = y.abs() * R.CHAIN + 2.0 ** -16
    R.assert_rounded(r.y, y, err, "y")
    assert_codes(r.codes.cpu(), r.scales.cpu(), y, err, qtype, mode)


@pytest.mark.parametrize("qtype", ["e4m3fn", "e5m2"])
def test_mx_exponents_next_to_a_power_of_two(qtype):
    """Blocks whose largest |y| lies within a few fp32 units of a power of two get the float64 value's exponent."""
    rows, H = 4000, 1024
    x, gamma = rnd(17, rows, H, std=2.0, mean=1.0), rnd(18, H, mean=1.0, std=0.3)
    beta = rnd(19, H, std=0.5)
    f = L.layer_norm(x, None, gamma, beta, 1e-5)
    r = binding.a2av_layer_norm(dev(x), dev(gamma), dev(beta), None, 1e-5, qtype, "mx")
    amax = f["y"].abs().unflatten(1, (-1, 32)).amax(2)
    want = (torch.floor(torch.log2(amax)) - R.F8[qtype][1]).long() + 127
    off = r.scales.cpu().long() != want
    m, _ = np.frexp(amax.numpy())
    near = torch.from_numpy(np.minimum(np.abs(2 * m - 1), np.abs(1 - m)))
    # a thread's sums of 8 products (the squares) and 16 values (the mean) stay in fp32
    assert float(near[off].max() if off.any() else 0.0) < 2.0 ** -26


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,H,with_dh", [(1, 8, True), (1, 7168, True), (7, 1000, False), (700, 256, True),
                                            (3000, 136, True), (650, 4096, False), (20, 9000, True), (20, 20000, True),
                                            (3, 65528, True), (9, 2048, True), (61, 4096, True), (128, 2048, False), (129, 2048, True),
                                            (32, 8192, True), (33, 8192, True), (256, 64, True), (20, 8200, True)])
def test_backward(rows, H, with_dh, dt):
    dtype = DT[dt]
    h, dy = rnd(20, rows, H, dtype=dtype, std=2.0, mean=1.0), rnd(21, rows, H, dtype=dtype, std=0.1)
    dh = rnd(22, rows, H, dtype=dtype, std=0.1) if with_dh else None
    gamma = rnd(23, H, dtype=dtype, std=0.2, mean=1.0)
    f = L.layer_norm(h, None, gamma, None, 1e-5)
    mean, rstd = f["mean"].float(), f["rstd"].float()
    dx, dgamma, dbeta = binding.a2av_layer_norm_backward(*dev(dy, h, gamma, mean, rstd, dh))
    rx, rg, rb = L.layer_norm_backward(dy, dh, h, gamma, mean, rstd)
    ex, eg, eb = L.gradient_bounds(dy, h, gamma, mean, rstd, rx)
    R.assert_rounded(dx, rx, ex, "dx")
    assert bool(((dgamma.cpu().double() - rg).abs() <= eg).all())
    assert bool(((dbeta.cpu().double() - rb).abs() <= eb).all())
    # in place over dh (or dy), and the same bits again
    over = dev(dh if with_dh else dy)
    args = (over if not with_dh else dev(dy), *dev(h, gamma, mean, rstd), over if with_dh else None)
    dx2, dg2, db2 = binding.a2av_layer_norm_backward(*args, dx=over)
    assert torch.equal(dx2.view(torch.int16), dx.view(torch.int16))
    assert torch.equal(dg2, dgamma) and torch.equal(db2, dbeta)


def test_backward_without_rows():
    z, none = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, device="cuda")
    dx, dgamma, dbeta = binding.a2av_layer_norm_backward(z, z, torch.ones(64, dtype=torch.bfloat16, device="cuda"), none,
                                                         none)
    assert dx.shape == (0, 64) and bool((dgamma == 0).all()) and bool((dbeta == 0).all())


@pytest.mark.parametrize("scale", [1e-30, 1e-4, 1e4, 1e30])
def test_backward_of_rows_of_any_scale(scale):
    h = (rnd(24, 30, 1024).float() * scale).bfloat16()
    dy, gamma = rnd(25, 30, 1024), rnd(26, 1024, mean=1.0, std=0.1)
    f = L.layer_norm(h, None, gamma, None, 0.0)
    mean, rstd = f["mean"].float(), f["rstd"].float()
    dx, _, _ = binding.a2av_layer_norm_backward(*dev(dy, h, gamma, mean, rstd))
    rx = L.layer_norm_backward(dy, None, h, gamma, mean, rstd)[0]
    R.assert_rounded(dx, rx, L.gradient_bounds(dy, h, gamma, mean, rstd, rx)[0], "dx")


def test_training_step_and_graph():
    """Forward and backward captured as one graph on a stream of its own give the eager calls' bits."""
    x, res, dy, dh = (rnd(30 + i, 777, 2056, dtype=torch.float16, std=0.5).cuda() for i in range(4))
    gamma, beta = rnd(35, 2056, dtype=torch.float16).cuda(), rnd(36, 2056, dtype=torch.float16).cuda()

    def step():
        f = binding.a2av_layer_norm(x, gamma, beta, res, want_stats=True)
        return (f.h, f.y, *binding.a2av_layer_norm_backward(dy, f.h, gamma, f.mean, f.rstd, dh))

    want = [t.clone() for t in step()]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        got = step()
    for t in got:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_squares_that_overflow_about_zero_only():
    # +-1.1e18 about 0.45e18: 256 squares sum to 3.6e38 about 0, beyond fp32, and to 3.1e38 about the mean.
    x = torch.full((2, 256), 1.55e18)
    x[:, ::2] = -0.65e18
    x, gamma, beta = x.to(torch.bfloat16), rnd(12, 256), rnd(13, 256)
    f = L.layer_norm(x, None, gamma, beta, 1e-5)
    assert float((x.double() ** 2).sum(1).max()) > torch.finfo(torch.float32).max
    assert float(((x.double() - f["mean"][:, None]) ** 2).sum(1).max()) < torch.finfo(torch.float32).max
    check(f, binding.a2av_layer_norm(dev(x), dev(gamma), dev(beta), eps=1e-5, want_stats=True, want_y=True), None, "mx",
          residual=False)


@pytest.mark.parametrize("qtype,mode", [("e4m3fn", "mx"), ("int8", "group128")])
@pytest.mark.parametrize("rows,H", [(700, 7168), (170, 16384), (200, 8192), (153, 8192), (2500, 512)])
def test_codes_around_the_limits_of_the_wide_weights(rows, H, qtype, mode):
    # One vector a thread while all rows are resident, then two with gamma and beta in shared memory, up to 128 KB.
    x, res = rnd(31, rows, H), rnd(32, rows, H)
    gamma, beta = rnd(33, H), rnd(34, H)
    for b in (beta, None):
        r = binding.a2av_layer_norm(dev(x), dev(gamma), dev(b), dev(res), eps=1e-5, qtype=qtype, mode=mode)
        check(L.layer_norm(x, res, gamma, b, 1e-5), r, qtype, mode, want_y=False)
