"""The grouped product of codes with a float32 scale per 128 on the GPU against float64 (needs a GB300).  Bounds:
tests/g128_ref.py."""

import ctypes

import numpy as np
import pytest
import torch

import ffn_ref as R
import g128_ref as G
from token_permute_grouped_gb300 import binding, build

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()


def inputs(seed, W, e, counts, K, N, qtype, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    A = int(sum(counts))
    size = torch.exp(spread * torch.randn(K, generator=g))
    x = torch.randn(A, K, generator=g) * size
    xq, xs = G.quantise(x, qtype, 1)
    wq, ws = G.quantise(torch.randn(e, N, K, generator=g) * K ** -0.5, qtype, 128)
    return xq, xs, torch.tensor(counts, dtype=torch.int32), wq, ws


def split(seed, W, e, sizes):
    """Counts [W * e] that give expert j sizes[j] rows, spread over the sources at random."""
    rng = np.random.default_rng(seed)
    c = np.stack([rng.multinomial(n, np.full(W, 1.0 / W)) for n in sizes], 1)
    return c.reshape(-1).tolist()


def guarded(A, N, dtype):
    """An output with values around it that no call may change."""
    pad = 64
    buf = torch.full((A * N + 2 * pad,), -7.0, dtype=dtype, device="cuda")
    return buf, buf[pad:pad + A * N].view(A, N)


def run(W, e, counts, K, N, dt, qtype, seed=1, spread=1.0):
    xq, xs, rc, wq, ws = inputs(seed, W, e, counts, K, N, qtype, spread)
    A = xq.shape[0]
    plan = binding.G128Plan(W, e, A, K, N, DT[dt], qtype)
    buf, y = guarded(A, N, DT[dt])
    args = [t.cuda() for t in (xq, xs, rc, wq, ws)]
    plan.run(*args, gmmY=y)
    assert binding.a2av_gmm_read_device_status(plan.workspace) == (0, 0)
    ref, err = G.product(xq, xs, counts, W, e, wq, ws, qtype)
    R.assert_rounded(y, ref, err, "y")
    assert bool((buf[:64] == -7.0).all()) and bool((buf[64 + A * N:] == -7.0).all())
    again = plan.run(*args)
    assert torch.equal(again.view(torch.int16), y.contiguous().view(torch.int16))
    return y


CASES = [  # W, e, rows of each expert, K, N
    (1, 1, [1], 128, 8), (1, 1, [1], 4096, 1024), (1, 1, [300], 256, 256), (1, 3, [5, 0, 9], 384, 72),
    (2, 2, [128, 128], 256, 128), (8, 4, [2, 3, 0, 3], 1024, 512), (4, 4, [33, 200, 1, 64], 1152, 328),
    (3, 5, [0, 400, 0, 257, 31], 640, 520), (16, 2, [700, 900], 512, 776), (1, 2, [0, 1500], 2048, 136),
    (2, 8, [150] * 8, 256, 1032), (8, 32, [40] * 32, 128, 264), (1, 1, [130], 7168, 256), (2, 1, [2600], 384, 2048),
]


@pytest.mark.parametrize("qtype", ["e4m3fn", "e5m2"])
@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("W,e,sizes,K,N", CASES)
def test_product(W, e, sizes, K, N, dt, qtype):
    run(W, e, split(7, W, e, sizes), K, N, dt, qtype)


@pytest.mark.parametrize("rows", [1, 2, 8, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129])
@pytest.mark.parametrize("W", [1, 4])
def test_few_rows_of_one_expert(rows, W):
    run(W, 3, split(8, W, 3, [0, rows, 1]), 768, 392, "bf16", "e4m3fn")


@pytest.mark.parametrize("W,e,sizes,K,N", [
    (1, 1, [1], 4096, 3080), (1, 1, [16], 2048, 6152), (3, 4, [0, 12, 0, 0], 2048, 1672), (5, 8, [0, 0, 30, 0, 0, 0, 0, 0], 1152, 1640),
    (2, 8, [1, 0, 3, 5, 0, 2, 16, 1], 1280, 1288), (4, 2, [7, 6], 7168, 1024), (8, 32, [1] * 32, 1024, 520), (1, 2, [0, 1], 128, 60000)])
@pytest.mark.parametrize("dt,qtype", [("bf16", "e4m3fn"), ("fp16", "e5m2")])
def test_few_rows_of_large_weights(W, e, sizes, K, N, dt, qtype):
    """Weights that take longest: streamed, the K blocks of all columns cut evenly over the SMs; rows as they spread at
    random, all at one expert, at experts between empty ones."""
    run(W, e, split(17, W, e, sizes), K, N, dt, qtype)


def test_few_rows_of_large_weights_inconsistent_counts():
    W, e, A, K, N = 2, 4, 8, 4096, 1024
    plan = binding.G128Plan(W, e, A, K, N)
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = lambda *s: torch.randint(0, 100, s, dtype=torch.uint8, device="cuda", generator=g)
    args = (codes(A, K), torch.ones(A, K // 128, device="cuda"))
    w = (codes(e, N, K), torch.ones(e, N // 128, K // 128, device="cuda"))
    counts = lambda *c: torch.tensor(c, dtype=torch.int32, device="cuda")
    good = counts(1, 1, 1, 1, 1, 1, 1, 1)
    want = plan.run(*args, good, *w)
    for bad in (counts(1, 1, 1, 1, 1, 1, 1, 2), counts(9, -1, 0, 0, 0, 0, 0, 0)):
        y = torch.full((A, N), 5.0, dtype=torch.bfloat16, device="cuda")
        plan.run(*args, bad, *w, gmmY=y)
        assert binding.STATUS_NAMES[binding.a2av_gmm_read_device_status(plan.workspace)[0]] == "A2AV_ERR_DEVICE_CHECK"
        assert bool((y == 5.0).all())
    plan.workspace.fill_(255)  # (nothing in it is kept from call to call)
    assert torch.equal(plan.run(*args, good, *w), want)
    assert binding.a2av_gmm_read_device_status(plan.workspace) == (0, 0)


def test_all_rows_at_one_of_many_experts():
    run(4, 16, split(9, 4, 16, [0] * 5 + [290] + [0] * 10), 512, 256, "bf16", "e4m3fn")


def test_without_rows():
    y = run(2, 2, [0, 0, 0, 0], 256, 64, "bf16", "e4m3fn")
    assert y.shape == (0, 64)


@pytest.mark.parametrize("sizes", [[3, 2], [400, 700]])
def test_special_values_stay_in_their_row_and_column(sizes):
    W, e, K, N = 2, 2, 512, 264
    counts = split(10, W, e, sizes)
    xq, xs, rc, wq, ws = inputs(11, W, e, counts, K, N, "e5m2")
    A = xq.shape[0]
    xs[0, 1] = float("nan")          # a row's block
    xq[1, 300] = 0x7f                # a NaN code
    xq[2, 7], xq[3 % A, 9] = 0x7c, 0xfc  # infinities
    xs[4 % A, 2] = 0.0               # a block of no size
    wq[1, 5, 17] = 0x7c              # an infinite weight: one column of expert 1
    ws[0, 1, 3] = float("inf")       # a block of columns of expert 0
    plan = binding.G128Plan(W, e, A, K, N, torch.bfloat16, "e5m2")
    y = plan.run(*[t.cuda() for t in (xq, xs, rc, wq, ws)])
    ref, err = G.product(xq, xs, counts, W, e, wq, ws, "e5m2")
    # An infinite scale meets sums of both signs: an infinity of the sums' sign or a NaN, as the sums come out.
    loose = torch.zeros(ref.shape, dtype=torch.bool)
    loose[:sum(counts[0::2]), 128:256] = True
    got = y.cpu().double()
    assert not bool(torch.isfinite(got[loose]).any())
    R.assert_rounded(torch.where(loose, torch.zeros_like(got), got).bfloat16(), ref.masked_fill(loose, 0.0),
                     err.masked_fill(loose, 0.0).nan_to_num(0.0, 0.0), "y")


@pytest.mark.parametrize("A", [40, 4000])
def test_inconsistent_counts_are_reported_and_nothing_is_written(A):
    xq, xs, rc, wq, ws = inputs(12, 2, 2, [A // 4] * 4, 256, 128, "e4m3fn")
    plan = binding.G128Plan(2, 2, A, 256, 128)
    for bad in ([A // 4] * 3 + [A // 4 + 1], [A, -1, 1, 0]):
        y = torch.full((A, 128), 5.0, dtype=torch.bfloat16, device="cuda")
        plan.run(xq.cuda(), xs.cuda(), torch.tensor(bad, dtype=torch.int32).cuda(), wq.cuda(), ws.cuda(), gmmY=y)
        status, _ = binding.a2av_gmm_read_device_status(plan.workspace)
        assert binding.STATUS_NAMES[status] == "A2AV_ERR_DEVICE_CHECK"
        assert bool((y == 5.0).all())
    plan.run(xq.cuda(), xs.cuda(), rc.cuda(), wq.cuda(), ws.cuda())
    assert binding.a2av_gmm_read_device_status(plan.workspace) == (0, 0)


def test_scales_that_start_anywhere():
    """float32 scales are 4-byte aligned, no more."""
    W, e, counts, K, N = 1, 1, [200], 384, 128
    xq, xs, rc, wq, ws = inputs(13, W, e, counts, K, N, "e4m3fn")
    xo, wo = torch.empty(xs.numel() + 1, device="cuda"), torch.empty(ws.numel() + 3, device="cuda")
    xo[1:], wo[3:] = xs.flatten().cuda(), ws.flatten().cuda()
    for A in (200, 3):
        plan = binding.G128Plan(W, e, A, K, N)
        y = plan.run(xq[:A].cuda(), xo[1:].view(xs.shape)[:A], torch.tensor([A], dtype=torch.int32).cuda(), wq.cuda(),
                     wo[3:].view(ws.shape))
        ref, err = G.product(xq[:A], xs[:A], [A], W, e, wq, ws, "e4m3fn")
        R.assert_rounded(y, ref, err, "y")


def test_offsets_past_2_31():
    """Rows and weights of more than 2^31 codes: rows of the last ones against float64."""
    K, N, A, e = 8192, 40960, 300_000, 8
    g = torch.Generator(device="cuda").manual_seed(3)
    xq = torch.randint(0, 120, (A, K), dtype=torch.uint8, device="cuda", generator=g)
    xs = torch.rand(A, K // 128, device="cuda", generator=g)
    wq = torch.randint(0, 120, (e, N, K), dtype=torch.uint8, device="cuda", generator=g)
    ws = torch.rand(e, N // 128, K // 128, device="cuda", generator=g) * 1e-3
    rc = torch.zeros(2 * e, dtype=torch.int32, device="cuda")
    rc[e - 1], rc[2 * e - 1] = 130, A - 130  # all at the last expert, its first rows from the first source
    rows = [0, 1, 129, 130, 262144, A - 1]
    plan = binding.G128Plan(2, e, A, K, N)
    y = plan.run(xq, xs, rc, wq, ws)
    cols = slice(N - 136, N)
    w = G.values(wq[-1, -256:], ws[-1, -2:], "e4m3fn", 128)[-136:]
    x = G.values(xq[rows], xs[rows], "e4m3fn")
    ref, mag = x @ w.t(), x.abs() @ w.abs().t()
    R.assert_rounded(y[rows][:, cols], ref, (136 + K // 128 + 1) * 2.0 ** -23 * mag, "y")
    few = binding.G128Plan(1, e, 3, K, N)
    rc = torch.zeros(e, dtype=torch.int32, device="cuda")
    rc[-1] = 3
    yf = few.run(xq[-3:].contiguous(), xs[-3:].contiguous(), rc, wq, ws)
    x = G.values(xq[-3:], xs[-3:], "e4m3fn")
    R.assert_rounded(yf[:, cols], x @ w.t(), (136 + K // 128 + 1) * 2.0 ** -23 * (x.abs() @ w.abs().t()), "few rows")
    torch.cuda.empty_cache()


def test_layer_in_eight_bits_and_graph():
    """Norm to codes, product, gated activation to codes, product, captured as one graph on a stream of its own."""
    W, e, K, N = 2, 2, 512, 256
    sizes = [70, 130]
    counts = split(14, W, e, sizes)
    A = sum(sizes)
    g = torch.Generator().manual_seed(15)
    x = torch.randn(A, K, generator=g).bfloat16().cuda()
    gamma = torch.ones(K, dtype=torch.bfloat16, device="cuda")
    gu, d = (G.quantise(torch.randn(*s, generator=g) * s[-1] ** -0.5, "e4m3fn", 128) for s in ((e, 2 * N, K), (e, K, N)))
    gu, d = [t.cuda() for t in gu], [t.cuda() for t in d]
    rc = torch.tensor(counts, dtype=torch.int32, device="cuda")
    per_expert = rc.view(W, e).sum(0, dtype=torch.int32)
    first, down = binding.G128Plan(W, e, A, K, 2 * N), binding.G128Plan(1, e, A, N, K)

    def layer():
        r = binding.a2av_layer_norm(x, gamma, qtype="e4m3fn", mode="group128")
        h = first.run(r.codes, r.scales, rc, *gu)
        q = binding.a2av_glu_quant(h, "silu", "e4m3fn", "group128")
        return r, h, q, down.run(q.codes, q.scales, per_expert, *d)

    r, h, q, y = layer()
    ref, err = G.product(r.codes.cpu(), r.scales, counts, W, e, gu[0], gu[1], "e4m3fn")
    R.assert_rounded(h, ref, err, "gate and up")
    ref, err = G.product(q.codes.cpu(), q.scales, sizes, 1, e, d[0], d[1], "e4m3fn")
    R.assert_rounded(y, ref, err, "down")
    torch.cuda.synchronize()
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph, stream=s):
        got = layer()[3]
    got.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, y)


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(seed):
    rng = np.random.default_rng([seed, 5])
    W, e = int(rng.choice([1, 2, 5, 8])), int(rng.choice([1, 2, 4, 7, 16]))
    A = int(np.exp(rng.uniform(0, np.log(3000))))
    counts = rng.multinomial(A, rng.dirichlet(np.full(W * e, 0.5))).tolist()
    K, N = 128 * int(rng.integers(1, 17)), 8 * int(rng.integers(1, 100))
    run(W, e, counts, K, N, str(rng.choice(["bf16", "fp16"])), str(rng.choice(["e4m3fn", "e5m2"])), seed)


def test_raw_call_on_another_stream():
    """The C entry on a stream of the caller's, from a workspace of exactly the size it asks for."""
    W, e, counts, K, N = 2, 2, [30, 40, 50, 60], 256, 136
    xq, xs, rc, wq, ws = [t.cuda() for t in inputs(16, W, e, counts, K, N, "e4m3fn")]
    desc = binding.G128Desc(W, e, 180, K, N, 1, 0)
    n = ctypes.c_size_t(0)
    lib = binding.load()
    assert lib.a2av_gmm_g128_workspace_size(ctypes.byref(desc), ctypes.byref(n)) == 0
    work = torch.empty(n.value, dtype=torch.uint8, device="cuda")
    y = torch.empty(180, N, dtype=torch.float16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    args = [t.data_ptr() for t in (xq, xs, rc, wq, ws, y, work)]
    assert lib.a2av_gmm_g128_run(ctypes.byref(desc), *args, n.value, s.cuda_stream) == 0
    s.synchronize()
    ref, err = G.product(xq, xs, counts, W, e, wq, ws, "e4m3fn")
    R.assert_rounded(y, ref, err, "y")
