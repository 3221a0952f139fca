"""The expert-layer operators on the GPU against float64 references (needs a GB300).  Bounds: tests/ffn_ref.py."""

import numpy as np
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


def rnd(seed, *shape, dtype=torch.bfloat16, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std + mean).to(dtype)


def dev(*ts):
    out = [None if t is None else t.cuda() for t in ts]
    return out[0] if len(out) == 1 else out


# ------------------------------------------------------------------ RMS norm


COMBOS = [(None, "mx"), ("e4m3fn", "mx"), ("e5m2", "mx"), ("e4m3fn", "group128"), ("e5m2", "group128"),
          ("int8", "group128")]


def check_norm(x, res, gamma, eps, qtype, mode, want_y, r):
    s, y, rstd = R.rms_norm(x, res, gamma, eps)
    if res is not None:
        R.assert_rounded(r.h, s, s.abs() * 2.0 ** -24, "h")
    if want_y:
        R.assert_rounded(r.y, y, y.abs() * R.CHAIN, "y")
    if qtype:
        R.assert_codes(r.codes, r.scales, y, R.CHAIN, qtype, mode, "codes")
    ok = torch.isfinite(rstd)
    assert bool(((r.rstd.cpu().double() - rstd).abs() <= R.CHAIN * rstd)[ok].all())


@pytest.mark.parametrize("qtype,mode", COMBOS)
@pytest.mark.parametrize("rows,H", [(1, 128), (1, 7168), (3, 256), (37, 1408), (200, 4096), (400, 2048), (5, 16512),
                                    (2, 34304), (3, 65408)])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_norm(rows, H, dt, qtype, mode):
    dtype = DT[dt]
    x, res = rnd(1, rows, H, dtype=dtype), rnd(2, rows, H, dtype=dtype, std=3.0)
    gamma = rnd(3, H, dtype=dtype, std=0.2, mean=1.0)
    r = binding.a2av_rms_norm(dev(x), dev(gamma), dev(res), 1e-5, qtype, mode, want_y=True, want_rstd=True)
    check_norm(x, res, gamma, 1e-5, qtype, mode, True, r)


@pytest.mark.parametrize("H", [8, 40, 136, 1000, 8200, 65528])
@pytest.mark.parametrize("rows", [1, 7, 300])
def test_norm_odd_widths(H, rows):
    x, gamma = rnd(4, rows, H, dtype=torch.float16), rnd(5, H, dtype=torch.float16)
    r = binding.a2av_rms_norm(dev(x), dev(gamma), None, 0.0, want_rstd=True)
    assert r.h is None and r.codes is None
    check_norm(x, None, gamma, 0.0, None, "mx", True, r)


def test_norm_only_codes_and_no_rows():
    x, gamma = rnd(6, 33, 512), rnd(7, 512)
    r = binding.a2av_rms_norm(dev(x), dev(gamma), qtype="e4m3fn")
    assert r.y is None and r.rstd is None
    R.assert_codes(r.codes, r.scales, R.rms_norm(x, None, gamma, 1e-6)[1], R.CHAIN, "e4m3fn", "mx", "codes")
    r = binding.a2av_rms_norm(dev(x)[:0], dev(gamma), qtype="e4m3fn", want_y=True)
    assert r.codes.shape == (0, 512) and r.y.shape == (0, 512)
    torch.cuda.synchronize()


def test_norm_strides_broadcast_and_in_place():
    wide, gamma = rnd(8, 50, 640), rnd(9, 512)
    x = wide.cuda()[:, 64:576]
    one = rnd(10, 1, 512)
    r = binding.a2av_rms_norm(x, dev(gamma), dev(one).expand(50, 512), 1e-6, "e5m2", "group128", want_y=True,
                              want_rstd=True)
    check_norm(wide[:, 64:576], one.expand(50, 512), gamma, 1e-6, "e5m2", "group128", True, r)
    # h in place of the residual, everything else into an earlier result's tensors
    res = rnd(11, 50, 512)
    buf = dev(res)
    again = binding.a2av_rms_norm(x, dev(gamma), buf, 1e-6, "e5m2", "group128", want_y=True, want_rstd=True,
                                  out=r._replace(h=buf))
    assert again.h.data_ptr() == buf.data_ptr() and again.codes.data_ptr() == r.codes.data_ptr()
    check_norm(wide[:, 64:576], res, gamma, 1e-6, "e5m2", "group128", True, again)


@pytest.mark.parametrize("qtype,mode", COMBOS[1:])
def test_norm_zero_and_non_finite_rows(qtype, mode):
    x, gamma = rnd(12, 8, 256), torch.ones(256, dtype=torch.bfloat16)
    x[1] = 0.0                       # a row of zeros: eps alone under the root
    x[3, 17] = float("nan")          # the whole row's statistics are NaN
    x[5, 200] = float("inf")         # rstd 0: inf * 0 is NaN there, zeros elsewhere
    x[6] = 3.3e38                    # finite, but its squares are not: rstd 0, every value 0
    gamma[40] = float("inf")         # one column's values infinite in every row
    r = binding.a2av_rms_norm(dev(x), dev(gamma), None, 1e-6, qtype, mode, want_y=True)
    s = x.float()
    with np.errstate(all="ignore"):
        rstd = torch.rsqrt((s * s).mean(1, keepdim=True) + 1e-6)
    y = (s * rstd * gamma.float()).double()
    R.assert_rounded(r.y, y, y.abs() * R.CHAIN, "y")
    R.assert_codes(r.codes, r.scales, y, R.CHAIN, qtype, mode, "codes")


@pytest.mark.parametrize("qtype,mode", COMBOS[1:])
def test_norm_tiny_and_huge_blocks(qtype, mode):
    # gamma carries the range: blocks near the smallest and the largest fp32 values, and a block of zeros.
    x = rnd(13, 4, 512)
    gamma = torch.ones(512, dtype=torch.bfloat16)
    gamma[:128], gamma[128:256], gamma[256:384] = 1e-38, 1e37, 0.0
    r = binding.a2av_rms_norm(dev(x), dev(gamma), None, 1e-6, qtype, mode)
    y = R.rms_norm(x, None, gamma, 1e-6)[1]
    R.assert_codes(r.codes, r.scales, y, R.CHAIN, qtype, mode, "codes")


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("rows,H,with_dh", [(1, 8, True), (1, 7168, True), (7, 1000, False), (700, 256, True),
                                            (3000, 136, True), (650, 4096, False), (20, 20000, True), (3, 65528, True)])
def test_norm_backward(rows, H, with_dh, dt):
    dtype = DT[dt]
    h, dy = rnd(14, rows, H, dtype=dtype, std=2.0), rnd(15, rows, H, dtype=dtype, std=0.1)
    dh = rnd(16, rows, H, dtype=dtype, std=0.1) if with_dh else None
    gamma = rnd(17, H, dtype=dtype, std=0.2, mean=1.0)
    rstd = R.rms_norm(h, None, gamma, 1e-6)[2].float()
    dx, dgamma = binding.a2av_rms_norm_backward(*dev(dy, h, gamma, rstd, dh))
    rx, rg = R.rms_norm_backward(dy, dh, h, gamma, rstd)
    n = h.double() * rstd.double()[:, None]
    a = dy.double() * gamma.double()
    # the row's mean adds H terms in fp32; every other step is one rounding
    err = R.CHAIN * rstd.double()[:, None] * (a.abs() + n.abs() * (a * n).abs().mean(1, keepdim=True)) + 2.0 ** -23 * rx.abs()
    R.assert_rounded(dx, rx, err, "dx")
    lim = (dy.double() * n).abs().sum(0) * (rows + 64) * 2.0 ** -24 + 1e-30
    assert bool(((dgamma.cpu().double() - rg).abs() <= lim).all())
    # in place over dh (or dy), and the same bits again
    over = dev(dh if with_dh else dy)
    args = (over if not with_dh else dev(dy), dev(h), dev(gamma), dev(rstd), over if with_dh else None)
    dx2, dg2 = binding.a2av_rms_norm_backward(*args, dx=over)
    assert torch.equal(dx2.view(torch.int16), dx.view(torch.int16)) and torch.equal(dg2, dgamma)


def test_norm_backward_without_rows():
    z = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    dx, dgamma = binding.a2av_rms_norm_backward(z, z, torch.ones(64, dtype=torch.bfloat16, device="cuda"),
                                                torch.empty(0, device="cuda"))
    assert dx.shape == (0, 64) and bool((dgamma == 0).all())


# ------------------------------------------------------------------ gated activation with codes


@pytest.mark.parametrize("qtype,mode", COMBOS)
@pytest.mark.parametrize("rows,N", [(1, 128), (37, 1408), (129, 512), (1000, 256)])
@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_glu_quant(rows, N, name, dt, qtype, mode):
    gu = rnd(20, rows, 2 * N, dtype=DT[dt], std=2.0)
    r = binding.a2av_glu_quant(dev(gu), name, qtype, mode, want_h=True)
    v = R.act(gu[:, :N].double(), name) * gu[:, N:].double()
    R.assert_rounded(r.h, v, v.abs() * R.CHAIN, "h")
    if qtype:
        R.assert_codes(r.codes, r.scales, v, R.CHAIN, qtype, mode, "codes")
        only = binding.a2av_glu_quant(dev(gu), name, qtype, mode)
        assert only.h is None and torch.equal(only.codes, r.codes)


def test_glu_quant_strided_rows_and_masked_values():
    wide = rnd(21, 21, 704, dtype=torch.float16)
    wide[3, 5] = float("inf")
    wide[4, 300] = float("nan")
    wide[5, 40:72] = -65504.0  # the type's lowest value: silu there is -0, a block of zeros
    r = binding.a2av_glu_quant(wide.cuda()[:, 8:520], "silu", "e4m3fn", "mx", want_h=True)
    gu = wide[:, 8:520]
    v = R.act(gu[:, :256].double(), "silu") * gu[:, 256:].double()
    # values below the smallest fp32 magnitude come out as zeros
    v = torch.where(v.abs() < 1e-37, torch.zeros_like(v), v)
    R.assert_rounded(r.h, v.where(v.abs() < 65504 * 2, v.sign() * float("inf")), v.abs() * R.CHAIN, "h")
    R.assert_codes(r.codes, r.scales, v, R.CHAIN, "e4m3fn", "mx", "codes")


@pytest.mark.parametrize("N", [8, 72])
def test_glu_without_codes_any_width(N):
    gu = rnd(22, 5, 2 * N)
    r = binding.a2av_glu_quant(dev(gu), "gelu_tanh", None)
    v = R.act(gu[:, :N].double(), "gelu_tanh") * gu[:, N:].double()
    R.assert_rounded(r.h, v, v.abs() * R.CHAIN, "h")


# ------------------------------------------------------------------ gated block and gradients


def counts_of(W, e, sizes, seed):
    """recvCounts whose experts have these row counts, split unevenly over the sources."""
    rng = np.random.default_rng(seed)
    c = np.zeros((W, e), np.int64)
    for j, n in enumerate(sizes):
        cuts = np.sort(rng.integers(0, n + 1, W - 1))
        c[:, j] = np.diff(np.concatenate([[0], cuts, [n]]))
    return c.reshape(-1).astype(np.int32)


BLOCKS = [
    # W, H1, N, rows of each expert
    (1, 64, 64, [1]),
    (1, 8, 8, [5]),
    (1, 128, 128, [256]),
    (1, 256, 128, [300, 20]),
    (2, 128, 136, [1, 0, 17, 129]),
    (3, 520, 328, [0, 0, 15, 16, 31, 127]),
    (4, 1032, 264, [255, 257, 3]),
    (8, 512, 704, [130, 64, 700, 0, 33]),
    (16, 192, 72, [40] * 16),
    (2, 2048, 320, [1000, 513]),
]


def _inputs(W, H1, N, sizes, dtype, seed=30):
    e, A = len(sizes), sum(sizes)
    counts = counts_of(W, e, sizes, seed)
    x = rnd(seed, A, H1, dtype=dtype)
    wg, wu = rnd(seed + 1, e, H1, N, dtype=dtype, std=H1 ** -0.5), rnd(seed + 2, e, H1, N, dtype=dtype, std=H1 ** -0.5)
    return e, A, counts, x, wg, wu


def _status(plan):
    return binding.a2av_gmm_read_device_status(plan.workspace)


@pytest.mark.parametrize("W,H1,N,sizes", BLOCKS)
@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_gated(W, H1, N, sizes, name, dt):
    dtype = DT[dt]
    e, A, counts, x, wg, wu = _inputs(W, H1, N, sizes, dtype)
    f = R.gated(x, counts, W, e, wg, wu, name)
    rc = torch.from_numpy(counts).cuda()
    xd, gd, ud = dev(x, wg, wu)
    # serving: nothing kept, rows read in place where they can be
    plan = binding.GatedPlan(W, e, A, H1, N, dtype, name)
    r = plan.run(xd, rc, gd, ud)
    assert _status(plan) == (0, 0)
    R.assert_rounded(r.h, f["h"], f["eh"], "h")
    # training
    plan = binding.GatedPlan(W, e, A, H1, N, dtype, name, save=True)
    t = plan.run(xd, rc, gd, ud)
    R.assert_rounded(t.h, f["h"], f["eh"], "h (kept)")
    assert torch.equal(t.permuteOut.cpu().view(torch.int16), x[f["idx"]].view(torch.int16))
    for got, ref, err in ((t.saved[0], f["G"], f["eg"]), (t.saved[1], f["U"], f["eu"])):
        assert bool(((got.cpu().double() - ref).abs() <= err).all())
    dh = rnd(40, A, N, dtype=dtype, std=0.5)
    b = plan.backward(dev(dh), t.permuteOut, rc, gd, ud, t.saved)
    assert _status(plan) == (0, 0)
    (dx, ex), ((dg, eg), (du, eu)) = R.gated_backward(f, dh, wg, wu, name, dtype)
    R.assert_rounded(b.dAtaOut, dx, ex, "dAtaOut")
    R.assert_rounded(b.dGate, dg, eg, "dGate")
    R.assert_rounded(b.dUp, du, eu, "dUp")
    # parts alone, and the same bits again
    only = plan.backward(dev(dh), t.permuteOut, rc, gd, ud, t.saved, want_weights=False)
    assert only.dGate is None and torch.equal(only.dAtaOut.view(torch.int16), b.dAtaOut.view(torch.int16))
    only = plan.backward(dev(dh), t.permuteOut, rc, gd, ud, t.saved, want_rows=False)
    assert only.dAtaOut is None and torch.equal(only.dUp.view(torch.int16), b.dUp.view(torch.int16))


@pytest.mark.parametrize("W,H1,N,sizes", BLOCKS)
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_gmm_backward(W, H1, N, sizes, dt):
    dtype = DT[dt]
    e, A, counts, x, w, _ = _inputs(W, H1, N, sizes, dtype, seed=50)
    dy = rnd(53, A, N, dtype=dtype, std=0.5)
    idx, _ = R.arrival_index(counts, W, e)
    xe = x[idx]
    plan = binding.GmmBackwardPlan(W, e, A, H1, N, dtype)
    dx, dw = plan.run(*dev(dy, xe, torch.from_numpy(counts), w))
    assert _status(plan) == (0, 0)
    (rx, ex), ((rw, ew),) = R.gmm_backward(xe, counts, W, e, dy, w)
    R.assert_rounded(dx, rx, ex, "dAtaOut")
    R.assert_rounded(dw, rw, ew, "dWeight")


@pytest.mark.parametrize("W,H1,N,sizes", [
    (1, 4096, 1024, [1]), (8, 4096, 1024, [3, 0, 4, 1]), (2, 8, 8, [1, 1]), (1, 1000, 72, [7]), (4, 520, 200, [0, 0, 0, 9]),
    (3, 2048, 136, [16]), (8, 264, 64, [1, 0, 2, 0, 1, 5, 3, 4]), (16, 7168, 320, [2] * 6), (1, 40, 1408, [8, 8]),
])
@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
def test_gated_few_rows(W, H1, N, sizes, name, dt):
    dtype = DT[dt]
    e, A, counts, x, wg, wu = _inputs(W, H1, N, sizes, dtype, seed=120)
    f = R.gated(x, counts, W, e, wg, wu, name)
    rc = torch.from_numpy(counts).cuda()
    guard = torch.full((A * N + 512,), 5.0, dtype=dtype, device="cuda")
    plan = binding.GatedPlan(W, e, A, H1, N, dtype, name, save=W == 1)
    r = plan.run(dev(x), rc, *dev(wg, wu), h=guard[:A * N].view(A, N))
    assert _status(plan) == (0, 0)
    R.assert_rounded(r.h, f["h"], f["eh"], "h")
    assert bool((guard[A * N:] == 5.0).all())
    if W == 1:
        for got, ref, err in ((r.saved[0], f["G"], f["eg"]), (r.saved[1], f["U"], f["eu"])):
            assert bool(((got.cpu().double() - ref).abs() <= err).all())


def test_gated_gradient_against_differences():
    """<gradient, direction> against central differences of the float64 forward."""
    W, H1, N, sizes, name = 2, 136, 72, [40, 0, 23], "silu"
    e, A, counts, x, wg, wu = _inputs(W, H1, N, sizes, torch.float16, seed=60)
    dh = rnd(63, A, N, dtype=torch.float16, std=0.5)
    plan = binding.GatedPlan(W, e, A, H1, N, torch.float16, name, save=True)
    rc = torch.from_numpy(counts).cuda()
    xd, gd, ud = dev(x, wg, wu)
    t = plan.run(xd, rc, gd, ud)
    b = plan.backward(dev(dh), t.permuteOut, rc, gd, ud, t.saved)
    f = R.gated(x, counts, W, e, wg, wu, name)
    (_, ex), ((_, eg), (_, eu)) = R.gated_backward(f, dh, wg, wu, name, torch.float16)
    loss = lambda x_, g_, u_: float((R.gated(x_, counts, W, e, g_, u_, name)["h"] * dh.double()).sum())
    base = [x.double(), wg.double(), wu.double()]
    for i, (grad, err) in enumerate(((b.dAtaOut, ex), (b.dGate, eg), (b.dUp, eu))):
        v = rnd(64 + i, *grad.shape, dtype=torch.float64)
        at = lambda s: loss(*[z + (s * v if k == i else 0) for k, z in enumerate(base)])
        diff = (at(1e-5) - at(-1e-5)) / 2e-5
        g = grad.double().cpu()
        lim = float(((err + R.U[torch.float16] * g.abs() + R.STEP[torch.float16]) * v.abs()).sum()) + 1e-4 * abs(diff)
        assert abs(float((g * v).sum()) - diff) <= lim, (i, diff)


def test_gated_no_rows():
    plan = binding.GatedPlan(2, 3, 0, 128, 64, save=True)
    rc = torch.zeros(6, dtype=torch.int32, device="cuda")
    w = rnd(70, 3, 128, 64).cuda()
    x = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    t = plan.run(x, rc, w, w)
    dh = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    ones = torch.ones(3, 128, 64, dtype=torch.bfloat16, device="cuda")
    b = plan.backward(dh, t.permuteOut, rc, w, w, t.saved, dGate=ones, dUp=ones.clone())
    assert _status(plan) == (0, 0)
    assert t.h.shape == (0, 64) and bool((b.dGate == 0).all()) and bool((b.dUp == 0).all())
    # the (empty) rows' gradient alone: nothing to write, and a status to read
    plan.workspace.fill_(0xff)
    b = plan.backward(dh, t.permuteOut, rc, w, w, t.saved, want_weights=False)
    assert b.dAtaOut.shape == (0, 128) and _status(plan) == (0, 0)
    m = binding.GmmBackwardPlan(2, 3, 0, 128, 64)
    m.workspace.fill_(0xff)
    dx, dw = m.run(dh, x, rc, w, want_weights=False)
    assert dx.shape == (0, 128) and dw is None and _status(m) == (0, 0)
    _, dw = m.run(dh, x, rc, w, want_rows=False)
    assert bool((dw == 0).all())


@pytest.mark.parametrize("W", [1, 3])
def test_non_finite_rows_stay_in_their_expert(W):
    """Infinities and NaN in one expert's rows reach neither another expert's rows nor its weights' gradients, on
    either side of a block that both share."""
    H1, N, sizes = 192, 136, [37, 19, 150, 5]
    e, A, counts, x, wg, wu = _inputs(W, H1, N, sizes, torch.bfloat16, seed=80)
    idx, _ = R.arrival_index(counts, W, e)
    dh = rnd(83, A, N, std=0.5)
    rc = torch.from_numpy(counts).cuda()

    def run(xe_bad):
        xa = x.clone()
        xa[idx[37:56]] = xe_bad  # all of expert 1's rows
        plan = binding.GatedPlan(W, e, A, H1, N, save=True)
        xd, gd, ud = dev(xa, wg, wu)
        t = plan.run(xd, rc, gd, ud)
        b = plan.backward(dev(dh), t.permuteOut, rc, gd, ud, t.saved)
        m = binding.GmmBackwardPlan(W, e, A, H1, N)
        dyb = dh.clone()
        dyb[37:56] = xe_bad
        dx, dw = m.run(dev(dyb), t.permuteOut, rc, gd)
        return [v.cpu() for v in (t.h, b.dAtaOut, b.dGate, b.dUp, dx, dw)]

    good, inf, nan = run(1.0), run(float("inf")), run(float("nan"))
    keep = torch.ones(A, dtype=torch.bool)
    keep[37:56] = False
    arrival = torch.zeros(A, dtype=torch.bool)
    arrival[idx] = keep
    others = [0, 2, 3]
    for bad in (inf, nan):
        for k, sel in enumerate((keep, arrival, others, others, arrival, others)):
            assert torch.equal(good[k][sel].view(torch.int16), bad[k][sel].view(torch.int16)), k
        assert not bool(torch.isfinite(bad[2][1].float()).all())


def test_inconsistent_counts_are_reported_and_nothing_is_written():
    W, H1, N, sizes = 2, 128, 64, [10, 20]
    e, A, counts, x, wg, wu = _inputs(W, H1, N, sizes, torch.bfloat16, seed=90)
    rc = torch.from_numpy(counts).cuda()
    rc[0] += 1
    plan = binding.GatedPlan(W, e, A, H1, N)
    h = torch.full((A, N), 7.0, dtype=torch.bfloat16, device="cuda")
    plan.run(dev(x), rc, dev(wg), dev(wu), h=h)
    assert binding.STATUS_NAMES[_status(plan)[0]] == "A2AV_ERR_DEVICE_CHECK"
    assert bool((h == 7.0).all())
    m = binding.GmmBackwardPlan(W, e, A, H1, N)
    dw = torch.full((e, H1, N), 7.0, dtype=torch.bfloat16, device="cuda")
    m.run(h, dev(x), rc, dev(wg), want_rows=False, dWeight=dw)
    assert binding.STATUS_NAMES[_status(m)[0]] == "A2AV_ERR_DEVICE_CHECK"
    assert bool((dw == 7.0).all())


def test_outputs_are_not_overrun():
    """Guard rows behind each output keep their pattern."""
    W, H1, N, sizes = 3, 136, 72, [33, 0, 130]
    e, A, counts, x, wg, wu = _inputs(W, H1, N, sizes, torch.bfloat16, seed=100)
    rc = torch.from_numpy(counts).cuda()
    dh = rnd(103, A, N)

    def guarded(*shape, dtype=torch.bfloat16):
        n = int(np.prod(shape))
        full = torch.full((n + 4096,), 5.0, dtype=dtype, device="cuda")
        return full, full[:n].view(*shape)

    full, outs = zip(*[guarded(A, N), guarded(2, A, N, dtype=torch.float32), guarded(A, H1), guarded(A, H1),
                       guarded(e, H1, N), guarded(e, H1, N)])
    plan = binding.GatedPlan(W, e, A, H1, N, save=True)
    xd, gd, ud = dev(x, wg, wu)
    t = plan.run(xd, rc, gd, ud, h=outs[0], saved=outs[1], permuteOut=outs[2])
    plan.backward(dev(dh), t.permuteOut, rc, gd, ud, t.saved, dAtaOut=outs[3], dGate=outs[4], dUp=outs[5])
    torch.cuda.synchronize()
    for f, o in zip(full, outs):
        assert bool((f[o.numel():] == 5.0).all())


def test_outputs_on_16_byte_boundaries():
    """Outputs and inputs that start 16 bytes into a 32-byte sector."""
    W, H1, N, sizes = 2, 128, 64, [300, 41]
    e, A, counts, x, wg, wu = _inputs(W, H1, N, sizes, torch.bfloat16, seed=130)
    rc = torch.from_numpy(counts).cuda()

    def off(t):
        buf = torch.empty(t.numel() + 8, dtype=t.dtype, device="cuda")
        return buf[8:].view(t.shape).copy_(t)

    f = R.gated(x, counts, W, e, wg, wu, "silu")
    dh = rnd(133, A, N)
    plan = binding.GatedPlan(W, e, A, H1, N, save=True)
    xd, gd, ud, dd = off(x), off(wg), off(wu), off(dh)
    t = plan.run(xd, rc, gd, ud, h=off(torch.zeros(A, N).bfloat16()), permuteOut=off(torch.zeros(A, H1).bfloat16()))
    R.assert_rounded(t.h, f["h"], f["eh"], "h")
    z = lambda *s: off(torch.zeros(*s).bfloat16())
    b = plan.backward(dd, t.permuteOut, rc, gd, ud, t.saved, dAtaOut=z(A, H1), dGate=z(e, H1, N), dUp=z(e, H1, N))
    (dx, ex), ((dg, eg), (du, eu)) = R.gated_backward(f, dh, wg, wu, "silu", torch.bfloat16)
    R.assert_rounded(b.dAtaOut, dx, ex, "dAtaOut")
    R.assert_rounded(b.dGate, dg, eg, "dGate")
    R.assert_rounded(b.dUp, du, eu, "dUp")
    few = binding.GatedPlan(1, e, 9, H1, N)
    rc9 = torch.tensor([4, 5], dtype=torch.int32, device="cuda")
    got = few.run(off(x[:9]), rc9, gd, ud, h=z(9, N)).h
    f = R.gated(x[:9], [4, 5], 1, e, wg, wu, "silu")
    R.assert_rounded(got, f["h"], f["eh"], "h (few rows)")


def test_earlier_results_are_written_again_only_where_they_fit():
    x, gamma = rnd(140, 6, 256).cuda(), rnd(141, 256).cuda()
    r = binding.a2av_rms_norm(x, gamma, x, qtype="e4m3fn")
    again = binding.a2av_rms_norm(x, gamma, x, qtype="e4m3fn", out=r)
    assert again.codes.data_ptr() == r.codes.data_ptr()
    with pytest.raises(ValueError, match="codes must be"):
        binding.a2av_rms_norm(x[:4], gamma, qtype="e4m3fn", out=r)
    with pytest.raises((TypeError, ValueError), match="scales must be"):
        binding.a2av_rms_norm(x, gamma, qtype="e4m3fn", mode="group128", out=r)
    y = binding.a2av_rms_norm(x, gamma, x, want_y=True, qtype="e4m3fn", out=r)
    assert y.y is not None and torch.equal(y.codes, again.codes)
    g = binding.a2av_glu_quant(x)
    assert binding.a2av_glu_quant(x, out=g).codes.data_ptr() == g.codes.data_ptr()
    with pytest.raises(ValueError, match="codes must be"):
        binding.a2av_glu_quant(x[:3], out=g)


@pytest.mark.parametrize("rows", [5, 400, 9000])  # few rows; one after the other; slopes beside the gradients' GEMM
def test_captured_in_a_graph(rows):
    """A layer's step captured once and replayed on new data gives what the calls give."""
    W, e, H1, N = 2, 2, 256, 128
    sizes = [rows - rows // 3, rows // 3]
    _, A, counts, x, wg, wu = _inputs(W, H1, N, sizes, torch.bfloat16, seed=150)
    rc = torch.from_numpy(counts).cuda()
    xd, gd, ud, gamma, dh = dev(x, wg, wu, rnd(153, H1), rnd(154, A, N))
    plan = binding.GatedPlan(W, e, A, H1, N, save=True)

    def step():
        n = binding.a2av_rms_norm(xd, gamma, want_y=True, want_rstd=True)
        t = plan.run(n.y, rc, gd, ud)
        b = plan.backward(dh, t.permuteOut, rc, gd, ud, t.saved)
        dx, dgamma = binding.a2av_rms_norm_backward(b.dAtaOut, xd, gamma, n.rstd)
        q = binding.a2av_glu_quant(t.h.view(A, N), qtype="e4m3fn")
        return [t.h, b.dGate, b.dUp, dx, dgamma, q.codes, q.scales]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for seed in (155, 156):
        xd.copy_(rnd(seed, A, H1))
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs]
        for a, b in zip(got, step()):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    assert _status(plan) == (0, 0)


def test_another_stream():
    W, H1, N, sizes = 2, 256, 128, [100, 60]
    e, A, counts, x, wg, wu = _inputs(W, H1, N, sizes, torch.bfloat16, seed=110)
    rc = torch.from_numpy(counts).cuda()
    xd, gd, ud = dev(x, wg, wu)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    plan = binding.GatedPlan(W, e, A, H1, N)
    ref = plan.run(xd, rc, gd, ud).h.clone()
    torch.cuda.synchronize()
    got = plan.run(xd, rc, gd, ud, stream=s).h
    with torch.cuda.stream(s):
        n = binding.a2av_rms_norm(got, torch.ones(N, dtype=torch.bfloat16, device="cuda"), qtype="e4m3fn")
    s.synchronize()
    assert torch.equal(got, ref)
    m = binding.a2av_rms_norm(ref, torch.ones(N, dtype=torch.bfloat16, device="cuda"), qtype="e4m3fn")
    assert torch.equal(n.codes, m.codes) and torch.equal(n.scales, m.scales)
