"""Alignments that include/a2av_ffn.h asks for: a pointer one step short of one is refused (no GPU needed: the calls return
before the library touches CUDA)."""

import pytest

import test_ffn_abi as C
from token_permute_grouped_gb300 import binding, build


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


@pytest.mark.parametrize("name,step", [("x", 8), ("residual", 8), ("gamma", 8), ("h", 8), ("y", 8), ("codes", 4), ("rstd", 2)])
def test_norm(lib, name, step):
    assert C.norm(lib, **{name: C.ptr(20) + step}) == C.UNSUPPORTED


@pytest.mark.parametrize("name,step", [("dy", 8), ("dh", 8), ("h", 8), ("gamma", 8), ("dx", 8), ("rstd", 2), ("dgamma", 8)])
def test_norm_backward(lib, name, step):
    assert C.norm_back(lib, **{name: C.ptr(20) + step}) == C.UNSUPPORTED


@pytest.mark.parametrize("name,step", [("gate", 8), ("up", 8), ("h", 8), ("codes", 4)])
def test_glu(lib, name, step):
    assert C.glu(lib, **{name: C.ptr(20) + step}) == C.UNSUPPORTED


def test_float_scales(lib):
    assert C.norm(lib, {"qmode": 1}, scales=C.ptr(20) + 2) == C.UNSUPPORTED
    assert C.glu(lib, {"qmode": 1}, scales=C.ptr(20) + 2) == C.UNSUPPORTED


@pytest.mark.parametrize("name,step", [("ataOut", 8), ("recvCounts", 2), ("gateWeight", 8), ("upWeight", 8),
                                       ("permuteOut", 8), ("h", 8), ("saved", 16)])
def test_gated_run(lib, name, step):
    assert C.gated_run(lib, **{name: C.ptr(20) + step}) == C.UNSUPPORTED


@pytest.mark.parametrize("name,step", [("dh", 8), ("permuteOut", 8), ("recvCounts", 2), ("gateWeight", 8), ("upWeight", 8),
                                       ("saved", 16), ("dAtaOut", 8), ("dGate", 8), ("dUp", 8)])
def test_gated_backward(lib, name, step):
    assert C.gated_back(lib, **{name: C.ptr(20) + step}) == C.UNSUPPORTED


@pytest.mark.parametrize("name,step", [("dY", 8), ("permuteOut", 8), ("recvCounts", 2), ("gmmWeight", 8), ("dAtaOut", 8),
                                       ("dWeight", 8)])
def test_gmm_backward(lib, name, step):
    assert C.gmm_back(lib, **{name: C.ptr(20) + step}) == C.UNSUPPORTED


def test_header_states_them():
    with open(build.INCLUDE + "/a2av_ffn.h") as f:
        text = " ".join(f.read().replace("*", " ").split())
    assert "dgamma 16-byte aligned" in text and "saved 32-byte" in text
