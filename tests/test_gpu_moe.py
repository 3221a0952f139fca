"""The expert layer for a few tokens on the GPU against float64 (needs a GB300).  Bounds: tests/moe_ref.py."""

import ctypes

import numpy as np
import pytest
import torch

import ffn_ref as R
import moe_ref as M
from token_permute_grouped_gb300 import binding, build

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()


def inputs(seed, T, E, H, N, dtype, router_dtype=None):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s, std=1.0: torch.randn(*s, generator=g) * std
    return {"x": rnd(T, H).to(dtype), "router": rnd(E, H, std=1.5 * H ** -0.5).to(router_dtype or dtype),
            "gate": rnd(E, H, N, std=H ** -0.5).to(dtype), "up": rnd(E, H, N, std=H ** -0.5).to(dtype),
            "down": rnd(E, N, H, std=N ** -0.5).to(dtype), "residual": rnd(T, H).to(dtype),
            "bias": rnd(E, std=0.1)}


def call(plan, s, bias=False, residual=True, **kw):
    d = {k: v.cuda() for k, v in s.items()}
    r = plan.run(d["x"], d["router"], d["gate"], d["up"], d["down"], bias=d["bias"] if bias else None,
                 residual=d["residual"] if residual else None, **kw)
    assert binding.a2av_gmm_read_device_status(plan.workspace) == (0, 0)
    return r


def check(r, s, K, act, dtype, bias=False, residual=True, **route):
    experts, w, ew, sure = M.route(s["x"], s["router"], K, bias=s["bias"] if bias else None, **route)
    got = r.experts.cpu().long()
    T, E = s["x"].shape[0], s["router"].shape[0]
    assert bool(((got >= 0) & (got < E)).all()) and all(len(set(row)) == K for row in got.tolist())
    assert torch.equal(got[sure], experts[sure])
    assert int(sure.sum()) * 2 >= T - 1  # most choices are beyond doubt
    gw = r.weights.cpu().double()
    assert bool(((gw - w).abs() <= ew * w.abs() + 1e-30)[sure].all())
    # the values follow from the weights that were given out
    y, err = M.values(s["x"], got, gw, torch.zeros_like(ew), s["gate"], s["up"], s["down"], act,
                      s["residual"] if residual else None, dtype)
    R.assert_rounded(r.y, y, err, "y")


CASES = [  # T, E, K, H, N
    (1, 1, 1, 8, 8), (1, 4, 2, 256, 128), (1, 32, 8, 1024, 512), (2, 3, 3, 136, 72), (3, 256, 8, 512, 64),
    (5, 31, 4, 1032, 328), (8, 8, 1, 64, 264), (16, 16, 2, 520, 136), (17, 7, 5, 2048, 200), (33, 40, 8, 264, 1032),
    (64, 64, 2, 392, 88), (64, 5, 3, 256, 640), (64, 2, 2, 128, 136), (64, 200, 8, 136, 72), (40, 1, 1, 640, 72),
]


@pytest.mark.parametrize("dt", ["bf16", "fp16"])
@pytest.mark.parametrize("T,E,K,H,N", CASES)
def test_layer(T, E, K, H, N, dt):
    s = inputs(1, T, E, H, N, DT[dt])
    plan = binding.MoePlan(T, E, K, H, N, DT[dt])
    r = call(plan, s)
    check(r, s, K, "silu", DT[dt])
    plan.workspace.fill_(255)  # (nothing in it is kept from call to call)
    again = call(plan, s)
    assert all(torch.equal(a, b) for a, b in zip(again, r))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalise", [True, False])
@pytest.mark.parametrize("bias", [True, False])
@pytest.mark.parametrize("router", [None, torch.float32])
def test_routing_forms(score, renormalise, bias, router):
    T, E, K, H, N = 23, 48, 6, 520, 72
    s = inputs(2, T, E, H, N, torch.float16, router)
    plan = binding.MoePlan(T, E, K, H, N, torch.float16, "gelu_tanh", score, renormalise, 2.5, router)
    check(call(plan, s, bias, residual=False), s, K, "gelu_tanh", torch.float16, bias, residual=False, score=score,
          renormalise=renormalise, scale=2.5)


@pytest.mark.parametrize("T", [9, 16, 17, 40, 64])
@pytest.mark.parametrize("E", [2, 64])
def test_every_token_at_the_same_experts(T, E):
    """The fullest expert has every token: several units of its rows where few were expected."""
    K, H, N = 2, 256, 136
    s = inputs(3, T, E, H, N, torch.bfloat16)
    s["bias"][:] = 0.0
    s["bias"][E - 1], s["bias"][0] = 20.0, 10.0
    plan = binding.MoePlan(T, E, K, H, N)
    r = call(plan, s, bias=True)
    assert bool((r.experts.cpu() == torch.tensor([E - 1, 0])).all())
    check(r, s, K, "silu", torch.bfloat16, bias=True)


def test_ties_go_to_the_lowest_index():
    T, E, K, H, N = 6, 20, 5, 64, 64
    s = inputs(4, T, E, H, N, torch.bfloat16)
    s["router"][:] = s["router"][0]
    s["x"][2] = 0.0
    r = call(binding.MoePlan(T, E, K, H, N), s)
    assert bool((r.experts.cpu() == torch.arange(K)).all())
    assert bool((r.weights.cpu() == 0.2).all())


def test_non_finite_values_stay_with_their_tokens():
    T, E, K, H, N = 12, 8, 2, 256, 72
    s = inputs(5, T, E, H, N, torch.bfloat16)
    clean = call(binding.MoePlan(T, E, K, H, N), s)
    chosen = clean.experts.cpu()
    broken = int(chosen[0, 0])
    s["x"][3] = float("nan")            # a token without a usable logit
    s["x"][7, 5] = float("inf")
    s["down"][broken, 3, 11] = float("inf")  # an expert's weights: what its tokens get is not finite
    s["gate"][broken, 0, 70] = float("nan")
    r = call(binding.MoePlan(T, E, K, H, N), s)
    hit = (chosen == broken).any(1)
    hit[3] = hit[7] = True
    assert not bool(torch.isfinite(r.y.cpu()[hit]).all(1).any())
    assert torch.equal(r.y.cpu()[~hit], clean.y.cpu()[~hit]) and bool((~hit).any())
    got = r.experts.cpu()
    assert bool(((got >= 0) & (got < E)).all()) and bool((got[:, 0] != got[:, 1]).all())
    assert torch.equal(got[3], torch.tensor([0, 1], dtype=torch.int32))  # all logits NaN: the lowest indices


def test_a_nan_logit_is_chosen_last():
    T, E, K, H, N = 2, 4, 4, 64, 64
    s = inputs(6, T, E, H, N, torch.bfloat16)
    s["router"][1, 3] = float("nan")
    r = call(binding.MoePlan(T, E, K, H, N), s)
    assert bool((r.experts.cpu()[:, 3] == 1).all())


def test_saturated_and_large_values():
    """Gated values beyond fp16's range go on as two summands; logits that differ by more than exp's range."""
    T, E, K, H, N = 4, 3, 2, 64, 64
    s = inputs(7, T, E, H, N, torch.float16)
    s["gate"] *= 30.0
    s["up"] *= 200.0
    s["down"] *= 1e-3
    s["router"] *= 100.0
    plan = binding.MoePlan(T, E, K, H, N, torch.float16)
    check(call(plan, s), s, K, "silu", torch.float16)


def test_in_place_no_tokens_and_another_stream():
    T, E, K, H, N = 5, 6, 2, 264, 72
    s = inputs(8, T, E, H, N, torch.bfloat16)
    plan = binding.MoePlan(T, E, K, H, N)
    want = call(plan, s)
    d = {k: v.cuda() for k, v in s.items()}
    w = (d["router"], d["gate"], d["up"], d["down"])
    over = d["residual"].clone()
    r = plan.run(d["x"], *w, residual=over, out=want._replace(y=over))
    assert r.y.data_ptr() == over.data_ptr()
    first = torch.equal(over, call(plan, s).y)
    over = d["x"].clone()
    plan.run(over, *w, residual=d["residual"], out=r._replace(y=over))
    assert first and torch.equal(over, call(plan, s).y)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    r = plan.run(d["x"], *w, residual=d["residual"], stream=stream)
    stream.synchronize()
    assert torch.equal(r.y, call(plan, s).y)
    none = binding.MoePlan(0, E, K, H, N)
    none.workspace.fill_(255)
    r = none.run(d["x"][:0], *w)
    assert r.y.shape == (0, H) and binding.a2av_gmm_read_device_status(none.workspace) == (0, 0)


def test_graph_and_two_calls_at_once():
    """A captured call replayed with new inputs; two plans on two streams at the same time, many times over."""
    T, E, K, H, N = 7, 32, 4, 512, 264
    a, b = inputs(9, T, E, H, N, torch.bfloat16), inputs(10, T, E, H, N, torch.bfloat16)
    plans = [binding.MoePlan(T, E, K, H, N) for _ in range(2)]
    want = [call(plans[0], a), call(plans[1], b)]
    dev = [{k: v.cuda() for k, v in s.items()} for s in (a, b)]
    run = lambda i, **kw: plans[i].run(dev[i]["x"], dev[i]["router"], dev[i]["gate"], dev[i]["up"], dev[i]["down"],
                                       residual=dev[i]["residual"], **kw)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    outs = [[], []]
    for _ in range(50):
        for i in range(2):
            outs[i].append(run(i, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o.y, want[i].y) and torch.equal(o.experts, want[i].experts) for o in outs[i])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        got = run(0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got.y, want[0].y)
    dev[0]["x"].copy_(dev[1]["x"])
    fresh = call(plans[1], {**a, "x": b["x"]}).y
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got.y, fresh)


def test_against_the_grouped_operators():
    """The same tokens through the gated block and the grouped product of the routed rows."""
    T, E, K, H, N = 11, 8, 2, 512, 256
    s = inputs(11, T, E, H, N, torch.bfloat16)
    r = call(binding.MoePlan(T, E, K, H, N), s, residual=False)
    ids = r.experts.cpu().long()
    order = torch.argsort(ids.flatten(), stable=True)
    counts = torch.bincount(ids.flatten(), minlength=E).to(torch.int32)
    rows = s["x"][order // K].cuda()
    plan = binding.GatedPlan(1, E, T * K, H, N)
    h = plan.run(rows, counts.cuda(), s["gate"].cuda(), s["up"].cuda()).h
    d = binding.Plan(1, E, T * K, N, H).run(h, counts.cuda(), s["down"].cuda())[0].float().cpu()
    y = torch.zeros(T, H).index_add_(0, order // K, d * r.weights.cpu().flatten()[order][:, None])
    # the chain rounds h and each expert's result to bf16
    assert float((r.y.cpu().float() - y).norm() / y.norm()) < 2 * 2.0 ** -8


def test_offsets_past_2_31():
    """Weights of more than 2^31 elements."""
    T, E, K, H, N = 2, 256, 2, 4096, 2112
    g = torch.Generator(device="cuda").manual_seed(12)
    rnd = lambda *sh: torch.randn(*sh, generator=g, device="cuda", dtype=torch.bfloat16)
    s = {"x": rnd(T, H), "router": rnd(E, H) * 0.02, "bias": torch.zeros(E, device="cuda")}
    s["gate"], s["up"], s["down"] = (torch.empty(E, *sh, dtype=torch.bfloat16, device="cuda") for sh in
                                     ((H, N), (H, N), (N, H)))
    for w in ("gate", "up", "down"):
        for e in range(E):
            s[w][e] = rnd(*s[w].shape[1:]) * s[w].shape[1] ** -0.5
    s["bias"][255], s["bias"][253] = 20.0, 10.0
    plan = binding.MoePlan(T, E, K, H, N)
    r = plan.run(s["x"], s["router"], s["gate"], s["up"], s["down"], bias=s["bias"])
    assert r.experts.tolist() == [[255, 253]] * T
    few = {k: v[252:].cpu() for k, v in s.items() if k in ("gate", "up", "down")}
    y, err = M.values(s["x"].cpu(), r.experts.cpu().long() - 252, r.weights.cpu().double(), torch.zeros(T, K), **few,
                      act="silu", residual=None, dtype=torch.bfloat16)
    R.assert_rounded(r.y, y, err, "y")
    torch.cuda.empty_cache()


@pytest.mark.parametrize("seed", range(20))
def test_random_shapes(seed):
    rng = np.random.default_rng([seed, 9])
    T, E = int(rng.integers(1, 65)), int(rng.integers(1, 80))
    K = int(rng.integers(1, min(E, 8) + 1))
    H, N = 8 * int(rng.integers(1, 80)), 8 * int(rng.integers(1, 50))
    dtype = DT[str(rng.choice(["bf16", "fp16"]))]
    act, score = str(rng.choice(["silu", "gelu_tanh"])), str(rng.choice(["softmax", "sigmoid"]))
    bias, residual, renorm = bool(rng.integers(2)), bool(rng.integers(2)), bool(rng.integers(2))
    s = inputs(100 + seed, T, E, H, N, dtype)
    plan = binding.MoePlan(T, E, K, H, N, dtype, act, score, renorm)
    check(call(plan, s, bias, residual), s, K, act, dtype, bias, residual, score=score, renormalise=renorm)


@pytest.mark.parametrize("T", [8, 9, 16, 17, 51, 64])
def test_jobs_of_many_shares(T):
    # A long contraction over a few columns, then a short one over many: what several CTAs have of a job is added, by
    # one of them and (second product, above 8 tokens) by a kernel behind it.
    s = inputs(21, T, 4, 3288, 192, torch.float16)
    plan = binding.MoePlan(T, 4, 4, 3288, 192, torch.float16, act="gelu_tanh")
    for residual in (True, False):
        r = call(plan, s, residual=residual)
        check(r, s, 4, "gelu_tanh", torch.float16, residual=residual)
    d = {k: v.cuda() for k, v in s.items()}
    want = plan.run(d["x"], d["router"], d["gate"], d["up"], d["down"], residual=d["x"])
    y = d["x"].clone()  # x, the residual and the result in one
    got = plan.run(y, d["router"], d["gate"], d["up"], d["down"], residual=y, out=binding.MoeOut(y, want.experts, want.weights))
    assert got.y.data_ptr() == y.data_ptr() and torch.equal(y, want.y)


@pytest.mark.parametrize("T,H", [(26, 384), (64, 136), (12, 8)])
def test_few_columns_of_many_experts(T, H):
    # All CTAs share the second product's one to three jobs.
    s = inputs(22, T, 49, H, 384, torch.bfloat16)
    plan = binding.MoePlan(T, 49, 7, H, 384)
    check(call(plan, s), s, 7, "silu", torch.bfloat16)


def test_two_plans_of_many_tokens_at_once_and_replayed():
    """Above 8 tokens a kernel behind the second product adds the shares: two streams at a time, and a graph of both."""
    T, E, K, H, N = 33, 24, 3, 264, 520
    plans = [binding.MoePlan(T, E, K, H, N) for _ in range(2)]
    hosts = [inputs(23 + i, T, E, H, N, torch.bfloat16) for i in range(2)]
    want = [call(plans[i], hosts[i]) for i in range(2)]
    dev = [{k: v.cuda() for k, v in s.items()} for s in hosts]
    run = lambda i, **kw: plans[i].run(dev[i]["x"], dev[i]["router"], dev[i]["gate"], dev[i]["up"], dev[i]["down"],
                                       residual=dev[i]["residual"], **kw)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for st in streams:
        st.wait_stream(torch.cuda.current_stream())
    outs = [[run(i, stream=streams[i]) for i in range(2)] for _ in range(40)]
    torch.cuda.synchronize()
    assert all(torch.equal(o[i].y, want[i].y) for o in outs for i in range(2))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=streams[0]):
        got = [run(0), run(1), run(0)]
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(g.y, want[i].y) for g, i in zip(got, (0, 1, 0)))
