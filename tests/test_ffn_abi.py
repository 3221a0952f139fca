"""Argument checks of the expert-layer operators' C ABI (include/a2av_ffn.h).  No GPU needed: every call here returns
before the library touches CUDA."""

import ctypes

import pytest
import torch

from token_permute_grouped_gb300 import binding, build

NAMES = binding.STATUS_NAMES
OK, NULLPTR, INVALID, UNSUPPORTED, WORKSPACE = ("A2AV_OK", "A2AV_ERR_NULLPTR", "A2AV_ERR_INVALID",
                                                "A2AV_ERR_UNSUPPORTED", "A2AV_ERR_WORKSPACE")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.load()


def ptr(i):
    return 0x100000 + 0x10000 * i


def norm(lib, desc=None, **kw):
    d = dict(rows=4, H=256, x_stride=256, residual_stride=256, dtype=0, qtype=0, qmode=0, eps=1e-6)
    d.update(desc or {})
    names = ["x", "residual", "gamma", "h", "y", "codes", "scales", "rstd"]
    args = [kw.get(n, ptr(i)) for i, n in enumerate(names)]
    return NAMES[lib.a2av_rms_norm(ctypes.byref(binding.RmsNormDesc(**d)), *args, None)]


@pytest.mark.parametrize("desc,kw,want", [
    ({"rows": -1}, {}, INVALID), ({"rows": 2 ** 31}, {}, INVALID), ({"H": 0}, {}, INVALID), ({"H": 65536}, {}, INVALID),
    ({"dtype": 2}, {}, INVALID), ({"eps": -1.0}, {}, INVALID), ({"eps": float("nan")}, {}, INVALID),
    ({"x_stride": 248}, {}, INVALID), ({"residual_stride": 8}, {}, INVALID), ({"x_stride": 260}, {}, UNSUPPORTED),
    ({"qtype": 3}, {}, INVALID), ({"qtype": 2}, {}, INVALID),       # INT8 has no mx form
    ({"qmode": 2}, {}, INVALID), ({"H": 264, "x_stride": 264, "residual_stride": 264}, {}, INVALID),
    ({"qmode": 1, "H": 160}, {}, INVALID),
    ({"H": 252, "qtype": -1}, {"codes": 0, "scales": 0}, UNSUPPORTED),
    ({}, {"x": 0}, NULLPTR), ({}, {"gamma": 0}, NULLPTR), ({}, {"codes": 0}, NULLPTR), ({}, {"scales": 0}, NULLPTR),
    ({"qtype": -1}, {}, INVALID),                                    # codes without a type
    ({"qtype": -1}, {"codes": 0, "scales": 0, "h": 0, "y": 0, "rstd": 0}, NULLPTR),
    ({}, {"x": ptr(0) + 8}, UNSUPPORTED), ({}, {"y": ptr(0) + 2}, UNSUPPORTED), ({}, {"codes": ptr(0) + 4}, UNSUPPORTED),
    ({"qmode": 1}, {"scales": ptr(0) + 2}, UNSUPPORTED), ({}, {"rstd": ptr(0) + 2}, UNSUPPORTED),
    ({"rows": 0}, {"x": 0, "residual": 0, "h": 0, "y": 0, "codes": 0, "scales": 0, "rstd": 0}, OK),
])
def test_norm_checks(lib, desc, kw, want):
    assert norm(lib, desc, **kw) == want


def test_norm_null_descriptor(lib):
    assert NAMES[lib.a2av_rms_norm(None, *[ptr(i) for i in range(8)], None)] == NULLPTR


def norm_back(lib, rows=400, H=256, dtype=0, wsbytes=1 << 20, **kw):
    names = ["dy", "dh", "h", "gamma", "rstd", "dx", "dgamma", "workspace"]
    args = [kw.get(n, ptr(i)) for i, n in enumerate(names)]
    return NAMES[lib.a2av_rms_norm_backward(rows, H, dtype, *args, wsbytes, None)]


@pytest.mark.parametrize("kw,want", [
    ({"rows": -1}, INVALID), ({"H": 0}, INVALID), ({"H": 65536}, INVALID), ({"dtype": 2}, INVALID),
    ({"H": 12}, UNSUPPORTED), ({"dy": 0}, NULLPTR), ({"h": 0}, NULLPTR), ({"gamma": 0}, NULLPTR), ({"rstd": 0}, NULLPTR),
    ({"dx": 0}, NULLPTR), ({"workspace": 0}, NULLPTR), ({"wsbytes": 16}, WORKSPACE), ({"workspace": ptr(9) + 16}, WORKSPACE),
    ({"dh": ptr(1) + 8}, UNSUPPORTED), ({"rows": 0, "dgamma": 0}, OK),
])
def test_norm_backward_checks(lib, kw, want):
    assert norm_back(lib, **kw) == want


def glu(lib, desc=None, **kw):
    d = dict(rows=4, N=256, stride=512, dtype=0, act=0, qtype=0, qmode=0)
    d.update(desc or {})
    args = [kw.get(n, ptr(i)) for i, n in enumerate(["gate", "up", "h", "codes", "scales"])]
    return NAMES[lib.a2av_glu_quant(ctypes.byref(binding.GluDesc(**d)), *args, None)]


@pytest.mark.parametrize("desc,kw,want", [
    ({"rows": -1}, {}, INVALID), ({"N": 0}, {}, INVALID), ({"stride": 248}, {}, INVALID), ({"act": 2}, {}, INVALID),
    ({"dtype": 2}, {}, INVALID), ({"qtype": 2}, {}, INVALID), ({"N": 264}, {}, INVALID), ({"stride": 516}, {}, UNSUPPORTED),
    ({}, {"gate": 0}, NULLPTR), ({}, {"up": 0}, NULLPTR), ({}, {"scales": 0}, NULLPTR),
    ({"qtype": -1}, {"codes": 0, "scales": 0, "h": 0}, NULLPTR), ({}, {"up": ptr(0) + 8}, UNSUPPORTED),
    ({"rows": 0}, {"gate": 0, "up": 0, "h": 0, "codes": 0, "scales": 0}, OK),
])
def test_glu_checks(lib, desc, kw, want):
    assert glu(lib, desc, **kw) == want


GATED = dict(W=2, e=4, A=1000, H1=512, N=256, dtype=0, act=0, want_permute_out=1, save=1)


def gated_size(lib, **kw):
    n = ctypes.c_size_t(0)
    d = binding.GatedDesc(**{**GATED, **kw})
    return NAMES[lib.a2av_gated_workspace_size(ctypes.byref(d), ctypes.byref(n))], n.value


@pytest.mark.parametrize("kw,want", [
    ({}, OK), ({"W": 0}, INVALID), ({"e": 33}, INVALID), ({"W": 65}, INVALID), ({"A": -1}, INVALID), ({"A": 2 ** 31}, INVALID),
    ({"H1": 65536}, INVALID), ({"N": 0}, INVALID), ({"dtype": 2}, INVALID), ({"act": 2}, INVALID),
    ({"H1": 508}, UNSUPPORTED), ({"N": 260}, UNSUPPORTED),
    ({"want_permute_out": 0}, INVALID),               # kept for a backward pass without the rows it reads
    ({"W": 1}, INVALID),                              # one source: the rows are expert-major already
    ({"W": 1, "want_permute_out": 0}, OK), ({"want_permute_out": 0, "save": 0}, OK),
])
def test_gated_descriptor(lib, kw, want):
    assert gated_size(lib, **kw)[0] == want


def test_gated_workspace(lib):
    # status, counts of finished pieces by 128 rows, then the larger of the staged rows and the two slopes
    pieces = (4 * (1000 // 128 + 1) + 255) // 256 * 256
    assert gated_size(lib)[1] == 256 + pieces + 2 * 1000 * 256 * 2
    assert gated_size(lib, A=32)[1] == 256 + 256 + 4 * 32 * 256 * 2  # each slope with what its rounding left over
    assert gated_size(lib, save=0)[1] == 256
    assert gated_size(lib, save=0, want_permute_out=0)[1] == 256 + 1000 * 512 * 2
    assert gated_size(lib, W=1, save=0, want_permute_out=0)[1] == 256
    assert gated_size(lib, A=0)[1] == 256


def gated_run(lib, desc=None, wsbytes=1 << 24, **kw):
    names = ["ataOut", "recvCounts", "gateWeight", "upWeight", "permuteOut", "h", "saved", "workspace"]
    args = [kw.get(n, ptr(i)) for i, n in enumerate(names)]
    return NAMES[lib.a2av_gated_run(ctypes.byref(binding.GatedDesc(**{**GATED, **(desc or {})})), *args, wsbytes, None)]


def gated_back(lib, desc=None, wsbytes=1 << 24, **kw):
    names = ["dh", "permuteOut", "recvCounts", "gateWeight", "upWeight", "saved", "dAtaOut", "dGate", "dUp", "workspace"]
    args = [kw.get(n, ptr(i)) for i, n in enumerate(names)]
    return NAMES[lib.a2av_gated_backward(ctypes.byref(binding.GatedDesc(**{**GATED, **(desc or {})})), *args, wsbytes,
                                         None)]


@pytest.mark.parametrize("name", ["ataOut", "recvCounts", "gateWeight", "upWeight", "permuteOut", "h", "saved", "workspace"])
def test_gated_run_pointers(lib, name):
    assert gated_run(lib, **{name: 0}) == NULLPTR
    assert gated_run(lib, **{name: ptr(20) + 2}) == (WORKSPACE if name == "workspace" else UNSUPPORTED)


def test_gated_run_refusals(lib):
    assert gated_run(lib, {"N": 260}) == UNSUPPORTED
    assert gated_run(lib, wsbytes=256) == WORKSPACE
    assert NAMES[lib.a2av_gated_run(None, *[ptr(i) for i in range(8)], 1 << 24, None)] == NULLPTR


@pytest.mark.parametrize("name", ["dh", "permuteOut", "recvCounts", "gateWeight", "upWeight", "saved", "workspace"])
def test_gated_backward_pointers(lib, name):
    assert gated_back(lib, **{name: 0}) == NULLPTR
    assert gated_back(lib, **{name: ptr(20) + 2}) == (WORKSPACE if name == "workspace" else UNSUPPORTED)


def test_gated_backward_refusals(lib):
    assert gated_back(lib, dGate=0) == NULLPTR                         # both weights' gradients or neither
    assert gated_back(lib, dAtaOut=0, dGate=0, dUp=0) == NULLPTR       # nothing asked for
    assert gated_back(lib, {"save": 0}) == INVALID
    assert gated_back(lib, wsbytes=1000) == WORKSPACE


def gmm_back(lib, desc=None, wsbytes=256, **kw):
    d = binding.make_desc(2, 4, 1000, 512, 256)
    for k, v in (desc or {}).items():
        setattr(d, k, v)
    names = ["dY", "permuteOut", "recvCounts", "gmmWeight", "dAtaOut", "dWeight", "workspace"]
    args = [kw.get(n, ptr(i)) for i, n in enumerate(names)]
    return NAMES[lib.a2av_gmm_backward(ctypes.byref(d), *args, wsbytes, None)]


@pytest.mark.parametrize("desc,kw,want", [
    ({"BS": 8, "H2": 64, "N2": 64}, {}, INVALID), ({"H1": 65536}, {}, INVALID), ({"N1": 252}, {}, UNSUPPORTED),
    ({}, {"dY": 0}, NULLPTR), ({}, {"permuteOut": 0}, NULLPTR), ({}, {"recvCounts": 0}, NULLPTR),
    ({}, {"gmmWeight": 0}, NULLPTR), ({}, {"workspace": 0}, NULLPTR), ({}, {"dAtaOut": 0, "dWeight": 0}, NULLPTR),
    ({}, {"dY": ptr(0) + 8}, UNSUPPORTED), ({}, {"recvCounts": ptr(0) + 2}, UNSUPPORTED), ({}, {"wsbytes": 128}, WORKSPACE),
])
def test_gmm_backward_checks(lib, desc, kw, want):
    kw = dict(kw)
    assert gmm_back(lib, desc, kw.pop("wsbytes", 256), **kw) == want


def test_binding_refuses_what_the_library_cannot_check():
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    with pytest.raises(TypeError, match="CUDA"):
        binding.a2av_rms_norm(x, x[0])
    with pytest.raises(TypeError, match="bfloat16 or float16"):
        binding.a2av_rms_norm(x.float(), x[0])
    with pytest.raises(TypeError, match="CUDA"):
        binding.a2av_glu_quant(x)
