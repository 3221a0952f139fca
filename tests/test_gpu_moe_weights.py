"""The weights of chosen experts whose scores lie below fp32's range, on the GPU: they are ratios, and a ratio of scores is in
range whatever the scores are.  Token t is 1 in place t, so that its logits are column t of the router."""

import pytest
import torch

import ffn_ref as R
import moe_ref as M
from token_permute_grouped_gb300 import binding, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()


def layer(logits, K, score, bias=None, renormalise=True, scale=1.0, dtype=torch.bfloat16):
    """Result and operands of a layer with these logits [T, E]."""
    logits = torch.tensor(logits, dtype=torch.float32)
    T, E = logits.shape
    H, N = 64, 72
    g = torch.Generator().manual_seed(1)
    router = torch.zeros(E, H)
    router[:, :T] = logits.t()
    s = {"x": torch.eye(T, H).to(dtype), "router": router}
    for name, shape in (("gate", (E, H, N)), ("up", (E, H, N)), ("down", (E, N, H))):
        s[name] = (torch.randn(*shape, generator=g) * 0.5).to(dtype)
    plan = binding.MoePlan(T, E, K, H, N, dtype, score=score, renormalise=renormalise, scale=scale, router_dtype=torch.float32)
    r = plan.run(*[t.cuda() for t in s.values()], bias=None if bias is None else torch.tensor(bias).cuda())
    assert binding.a2av_gmm_read_device_status(plan.workspace) == (0, 0)
    return r, s, logits.double()


def check(r, s, logits, experts, score, scale=1.0):
    """Choice, weights within an fp32 chain (and the exponent's own rounding: its difference of logits is good to 2^-24 of
    them), and values that follow from the weights."""
    got = r.experts.cpu().long()
    assert torch.equal(got, torch.tensor(experts))
    chosen = logits.gather(1, got)
    w = torch.softmax(chosen if score == "softmax" else torch.nn.functional.logsigmoid(chosen), 1) * scale
    gw = r.weights.cpu().double()
    assert bool(((gw - w).abs() <= R.CHAIN * w.abs() + 1e-30).all()), (gw, w)
    y, err = M.values(s["x"], got, gw, torch.zeros_like(gw), s["gate"], s["up"], s["down"], "silu", None, s["x"].dtype)
    R.assert_rounded(r.y, y, err, "y")


def test_sigmoid_scores_below_the_range():
    logits = [[-95.0, -96.5, -97.0, -120.0, -130.0, -95.5], [-10000.0, -10001.0, -10000.5, -10100.0, -2e4, -3e4],
              [-88.0, -89.0, -90.0, -91.0, -87.5, -86.0], [5.0, -200.0, -100.0, -300.0, -400.0, -500.0],
              [-0.5, 0.5, -2.0, -1.0, -3.0, -4.0], [-1e-3, 0.0, -80.0, -0.5, -1.0, -60.0], [-3e38, -1e30, -1e38, -2e30, -3e30, -2e38],
              [-700.0, -1.0, -90.0, -200.0, -3.0, -1000.0]]
    experts = [sorted(range(6), key=lambda e: -row[e])[:3] for row in logits]
    for dtype in (torch.bfloat16, torch.float16):
        r, s, l = layer(logits, 3, "sigmoid", scale=2.5, dtype=dtype)
        check(r, s, l, experts, "sigmoid", 2.5)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_a_bias_that_chooses_experts_far_below_the_largest_logit(score):
    logits = [[0.0, -120.0, -121.0, -250.0, -1.0], [0.0, -500.0, -500.25, 0.0, -1.0], [20.0, -3.0, -2.0, 1.0, -1.0],
              [100.0, -60.0, -300.0, 5.0, -1.0], [-2.0, -130.0, -131.0, -1.0, -3.0]]
    bias = [0.0, 6.0, 4.0, 0.0, 0.0]
    r, s, l = layer(logits, 2, score, bias)
    check(r, s, l, [[1, 2]] * 5, score)


def test_a_softmax_over_a_logit_that_is_not_a_number_has_no_weights():
    """Chosen or not, a NaN or +infinity among a token's logits leaves no softmax; an expert at -infinity has none of it."""
    nan, inf = float("nan"), float("inf")
    logits = [[1.0, nan, 0.0, -1.0], [1.0, inf, 0.0, -1.0], [1.0, -1e38, 0.0, -1.0]]
    # (one-hot tokens would meet 0 x infinity in the others' columns: one token a call)
    for renormalise in (True, False):
        for t, row in enumerate(logits):
            r, _, _ = layer([row], 2, "softmax", renormalise=renormalise)
            assert bool(torch.isnan(r.weights).any()) == (t < 2)
    r, s, l = layer([logits[2]], 2, "softmax")
    check(r, s, l, [[0, 2]], "softmax")
