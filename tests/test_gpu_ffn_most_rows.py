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


# Two sources, two experts: the last segment starts inside the last 128-row block of its expert.
COUNTS = [700_000_001, 747_483_596, 699_999_999, 51]


def places():
    """(first arrival row, first expert-major row, rows, expert) of each segment, expert-major."""
    starts = [sum(COUNTS[:i]) for i in range(4)]
    out, at = [], 0
    for place, seg in enumerate((0, 2, 1, 3)):
        out.append((starts[seg], at, COUNTS[seg], place // 2))
        at += COUNTS[seg]
    return out


def assert_rows(got, want, from_row, rows, repeats_at):
    """got's rows from from_row on are want's, which repeat, from row repeats_at of the repetition on."""
    same = torch.ones((), dtype=torch.bool, device=DEV)
    done = 0
    while done < rows:
        first = (repeats_at + done) % BLOCK
        n = min(BLOCK - first, rows - done)
        same &= (got[from_row + done:from_row + done + n] == want[first:first + n]).all()
        done += n
    assert bool(same)


def test_gated_block():
    assert sum(COUNTS) == ROWS
    block, wg, wu = rnd(3, BLOCK, H).to(DEV), rnd(4, 2, H, H).to(DEV), rnd(5, 2, H, H).to(DEV)
    one = []
    for j in range(2):
        plan = binding.GatedPlan(1, 1, BLOCK, H, H)
        rc = torch.tensor([BLOCK], dtype=torch.int32, device=DEV)
        one.append(plan.run(block, rc, wg[j:j + 1], wu[j:j + 1]).h)
        f = R.gated(block[:2048].cpu(), [2048], 1, 1, wg[j:j + 1].cpu(), wu[j:j + 1].cpu(), "silu")
        R.assert_rounded(one[j][:2048], f["h"], f["eh"], "h")
    plan = binding.GatedPlan(2, 2, ROWS, H, H)
    h = plan.run(repeated(block), torch.tensor(COUNTS, dtype=torch.int32, device=DEV), wg, wu).h
    assert binding.a2av_gmm_read_device_status(plan.workspace) == (0, 0)
    for arrival, place, rows, j in places():
        assert_rows(h, one[j], place, rows, arrival)


def test_gmm_backward_rows():
    dy, w = rnd(6, BLOCK, H).to(DEV), rnd(7, 2, H, H).to(DEV)
    one = []
    for j in range(2):
        plan = binding.GmmBackwardPlan(1, 1, BLOCK, H, H)
        rc = torch.tensor([BLOCK], dtype=torch.int32, device=DEV)
        one.append(plan.run(dy, dy, rc, w[j:j + 1], want_weights=False)[0])
        (rx, ex), _ = R.gmm_backward(dy[:2048].cpu(), [2048], 1, 1, dy[:2048].cpu(), w[j:j + 1].cpu())
        R.assert_rounded(one[j][:2048], rx, ex, "dAtaOut")
    big = repeated(dy)
    plan = binding.GmmBackwardPlan(2, 2, ROWS, H, H)
    dx, _ = plan.run(big, big, torch.tensor(COUNTS, dtype=torch.int32, device=DEV), w, want_weights=False)
    assert binding.a2av_gmm_read_device_status(plan.workspace) == (0, 0)
    for arrival, place, rows, j in places():
        assert_rows(dx, one[j], arrival, rows, place)


def test_gmm_backward_weights():
    """Rows of small whole numbers, mostly zeros, so that every sum is exact in fp32."""
    block = torch.zeros(BLOCK, H, dtype=torch.bfloat16)
    block[::16384] = torch.randint(-2, 3, (64, H), generator=torch.Generator().manual_seed(8)).bfloat16()
    block[-1] = 1.0
    x = repeated(block.to(DEV))
    x[-50:] = 2.0  # of the last expert's last segment
    plan = binding.GmmBackwardPlan(2, 2, ROWS, H, H)
    rc = torch.tensor(COUNTS, dtype=torch.int32, device=DEV)
    _, dw = plan.run(x, x, rc, rnd(9, 2, H, H).to(DEV), want_rows=False)
    assert binding.a2av_gmm_read_device_status(plan.workspace) == (0, 0)
    cut = COUNTS[0] + COUNTS[2]  # the experts' rows: [0, cut) and [cut, ROWS)
    for j, (a, z) in enumerate(((0, cut), (cut, ROWS))):
        ref = torch.zeros(H, H, dtype=torch.float64, device=DEV)
        for at in range(a, z, 2 ** 26):
            part = x[at:min(at + 2 ** 26, z)].double()
            ref += part.t() @ part
        assert torch.equal(dw[j].double(), ref.bfloat16().double())
