"""Argument checks of the product of codes with a float32 scale per 128 (no GPU needed: every call returns before the
library touches CUDA)."""

import ctypes

import pytest
import torch

from token_permute_grouped_gb300 import binding, build

NAMES = binding.STATUS_NAMES
OK, NULLPTR, INVALID, UNSUPPORTED, WORKSPACE = ("A2AV_OK", "A2AV_ERR_NULLPTR", "A2AV_ERR_INVALID",
                                                "A2AV_ERR_UNSUPPORTED", "A2AV_ERR_WORKSPACE")
DESC = dict(W=2, e=2, A=100, H1=256, N1=64, dtype=0, qtype=0)


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def ptr(i):
    return 0x100000 + 0x10000 * i


def size(lib, **desc):
    n = ctypes.c_size_t(0)
    st = lib.a2av_gmm_g128_workspace_size(ctypes.byref(binding.G128Desc(**{**DESC, **desc})), ctypes.byref(n))
    return NAMES[st], n.value


def run(lib, desc=None, wsbytes=1 << 20, **kw):
    names = ["ataOut_q", "ataOut_s", "recvCounts", "gmmWeight_q", "gmmWeight_s", "gmmY", "workspace"]
    args = [kw.get(n, ptr(i)) for i, n in enumerate(names)]
    return NAMES[lib.a2av_gmm_g128_run(ctypes.byref(binding.G128Desc(**{**DESC, **(desc or {})})), *args, wsbytes, None)]


BAD = [({"W": 0}, INVALID), ({"e": 0}, INVALID), ({"e": 33}, INVALID), ({"W": 129}, INVALID), ({"A": -1}, INVALID),
       ({"A": 2 ** 31}, INVALID), ({"H1": 0}, INVALID), ({"H1": 65536}, INVALID), ({"N1": 0}, INVALID),
       ({"N1": 65536}, INVALID), ({"dtype": 2}, INVALID), ({"qtype": 2}, INVALID), ({"qtype": -1}, INVALID),
       ({"H1": 192}, UNSUPPORTED), ({"N1": 12}, UNSUPPORTED)]


@pytest.mark.parametrize("desc,want", BAD)
def test_descriptor(lib, desc, want):
    assert size(lib, **desc)[0] == want
    assert run(lib, desc) == want


@pytest.mark.parametrize("kw,want", [
    *[({n: 0}, NULLPTR) for n in ("ataOut_q", "ataOut_s", "recvCounts", "gmmWeight_q", "gmmWeight_s", "gmmY", "workspace")],
    ({"ataOut_q": ptr(0) + 8}, UNSUPPORTED), ({"gmmWeight_q": ptr(0) + 8}, UNSUPPORTED), ({"gmmY": ptr(0) + 8}, UNSUPPORTED),
    ({"ataOut_s": ptr(0) + 2}, UNSUPPORTED), ({"gmmWeight_s": ptr(0) + 2}, UNSUPPORTED),
    ({"recvCounts": ptr(0) + 2}, UNSUPPORTED), ({"workspace": ptr(0) + 64}, WORKSPACE), ({"wsbytes": 255}, WORKSPACE),
])
def test_pointers(lib, kw, want):
    assert run(lib, **kw) == want


def test_null_descriptor_and_sizes(lib):
    n = ctypes.c_size_t(0)
    assert NAMES[lib.a2av_gmm_g128_workspace_size(None, ctypes.byref(n))] == NULLPTR
    assert NAMES[lib.a2av_gmm_g128_workspace_size(ctypes.byref(binding.G128Desc(**DESC)), None)] == NULLPTR
    assert NAMES[lib.a2av_gmm_g128_run(None, *[ptr(i) for i in range(7)], 1 << 20, None)] == NULLPTR
    st, several = size(lib)
    assert st == OK and several >= 256 + 100 * 256  # the staged rows
    assert size(lib, W=1)[0] == OK


def test_plan_refuses_types():
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        binding.G128Plan(1, 1, 4, 256, 64, torch.float32)
    with pytest.raises(ValueError, match="qtype"):
        binding.G128Plan(1, 1, 4, 256, 64, qtype="fp4")
    with pytest.raises(binding.A2avError, match="INVALID"):
        binding.G128Plan(1, 1, 4, 256, 64, qtype="int8", device="cpu")
