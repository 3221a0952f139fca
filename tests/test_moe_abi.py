"""Argument checks of the expert layer for a few tokens (no GPU needed: every call returns before the library touches
CUDA)."""

import ctypes

import pytest
import torch

from token_permute_grouped_gb300 import binding, build

NAMES = binding.STATUS_NAMES
OK, NULLPTR, INVALID, UNSUPPORTED, WORKSPACE = ("A2AV_OK", "A2AV_ERR_NULLPTR", "A2AV_ERR_INVALID",
                                                "A2AV_ERR_UNSUPPORTED", "A2AV_ERR_WORKSPACE")
DESC = dict(T=4, E=8, K=2, H=256, N=64, dtype=0, router_dtype=0, act=0, score=0, renormalise=1, scale=1.0)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def ptr(i):
    return 0x100000 + 0x10000 * i


def size(lib, **desc):
    n = ctypes.c_size_t(0)
    st = lib.a2av_moe_workspace_size(ctypes.byref(binding.MoeDesc(**{**DESC, **desc})), ctypes.byref(n))
    return NAMES[st], n.value


def run(lib, desc=None, wsbytes=1 << 24, **kw):
    names = ["x", "router", "bias", "gate", "up", "down", "residual", "y", "experts", "weights", "workspace"]
    args = [kw.get(n, ptr(i)) for i, n in enumerate(names)]
    return NAMES[lib.a2av_moe_run(ctypes.byref(binding.MoeDesc(**{**DESC, **(desc or {})})), *args, wsbytes, None)]


@pytest.mark.parametrize("desc,want", [
    ({"T": -1}, INVALID), ({"T": 65}, INVALID), ({"E": 0}, INVALID), ({"E": 257}, INVALID), ({"K": 0}, INVALID),
    ({"K": 9, "E": 16}, INVALID), ({"K": 3, "E": 2}, INVALID), ({"H": 0}, INVALID), ({"H": 65536}, INVALID),
    ({"N": 0}, INVALID), ({"N": 65536}, INVALID), ({"dtype": 2}, INVALID), ({"router_dtype": 1}, INVALID),
    ({"router_dtype": 3}, INVALID), ({"act": 2}, INVALID), ({"score": 2}, INVALID), ({"scale": float("nan")}, INVALID),
    ({"scale": float("inf")}, INVALID), ({"H": 260}, UNSUPPORTED), ({"N": 60}, UNSUPPORTED)])
def test_descriptor(lib, desc, want):
    assert size(lib, **desc)[0] == want
    assert run(lib, desc) == want


@pytest.mark.parametrize("kw,want", [
    *[({n: 0}, NULLPTR) for n in ("x", "router", "gate", "up", "down", "y", "workspace")],
    *[({n: ptr(0) + 8}, UNSUPPORTED) for n in ("x", "router", "bias", "gate", "up", "down", "residual", "y")],
    ({"experts": ptr(0) + 2}, UNSUPPORTED), ({"weights": ptr(0) + 1}, UNSUPPORTED),
    ({"workspace": ptr(0) + 64}, WORKSPACE), ({"wsbytes": 256}, WORKSPACE),
])
def test_pointers(lib, kw, want):
    assert run(lib, **kw) == want


def test_null_descriptor_and_sizes(lib):
    n = ctypes.c_size_t(0)
    assert NAMES[lib.a2av_moe_workspace_size(None, ctypes.byref(n))] == NULLPTR
    assert NAMES[lib.a2av_moe_workspace_size(ctypes.byref(binding.MoeDesc(**DESC)), None)] == NULLPTR
    assert NAMES[lib.a2av_moe_run(None, *[ptr(i) for i in range(11)], 1 << 20, None)] == NULLPTR
    # at least the logits, and the gated values of every choice in two summands
    st, n = size(lib)
    assert st == OK and n >= 256 + 4 * 8 * 4 + 4 * 2 * 64 * 4
    assert size(lib, router_dtype=2)[0] == OK and size(lib, T=0)[0] == OK


def test_plan_refuses_types():
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        binding.MoePlan(1, 4, 2, 256, 64, torch.float32)
    with pytest.raises(TypeError, match="router_dtype"):
        binding.MoePlan(1, 4, 2, 256, 64, torch.float16, router_dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="score"):
        binding.MoePlan(1, 4, 2, 256, 64, score="argmax")
    with pytest.raises(ValueError, match="act"):
        binding.MoePlan(1, 4, 2, 256, 64, act="relu")
    plan = binding.MoePlan(1, 4, 2, 256, 64, device="cpu")
    with pytest.raises(TypeError, match="CUDA"):
        plan.run(*[torch.zeros(1)] * 5)
