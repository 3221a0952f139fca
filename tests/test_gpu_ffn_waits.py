"""Waits of the expert-layer kernels that run out, each with a limit of milliseconds (on the GPU): a warp leaves such a wait
as one, and a kernel whose wait ran out reports it and leaves the GPU usable."""

import ctypes
import os
import subprocess

import pytest
import torch

from token_permute_grouped_gb300 import binding, build

pytestmark = pytest.mark.gpu

DEV = "cuda:0"
TIMEOUT = 2  # kStatusTimeout of csrc/plan.cuh


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build(checks=True)


def test_a_warp_leaves_a_wait_as_one(tmp_path):
    src, so = os.path.join(os.path.dirname(__file__), "wait_probe.cu"), str(tmp_path / "probe.so")
    subprocess.run([build.nvcc(), *build.ARCH, "-O3", "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-I", build.CSRC, "-I",
                    build.INCLUDE, src, "-o", so], check=True)
    probe = ctypes.CDLL(so).run_probe
    probe.argtypes = [ctypes.c_void_p, ctypes.c_void_p, ctypes.c_uint64, ctypes.c_void_p]
    out = torch.full((64,), -1, dtype=torch.int32, device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    assert probe(out.data_ptr(), status.data_ptr(), 5_000_000, torch.cuda.current_stream().cuda_stream) == 0
    assert out[:32].tolist() == [0] * 32   # some lanes' phase had completed; none of them goes on
    assert out[32:].tolist() == [1] * 32   # a completed phase, to all
    assert int(status) == TIMEOUT


@pytest.mark.parametrize("W,sizes", [(1, [9001]), (3, [5003, 0, 17, 1, 4101])])
def test_slopes_that_never_come(W, sizes):
    """The gradients' GEMM waits for one more piece of the slopes than there is."""
    e, A, H1, N = len(sizes), sum(sizes), 1536, 1448
    assert A * H1 * N >= 2e10  # slopes are computed beside the GEMM
    g = torch.Generator(device=DEV).manual_seed(1)
    rnd = lambda *s, std=1.0: torch.empty(*s, dtype=torch.bfloat16, device=DEV).normal_(0.0, std, generator=g)
    counts = torch.zeros(W, e, dtype=torch.int32)
    counts[0] = torch.tensor(sizes) // W
    for w in range(1, W):
        counts[w] = torch.tensor(sizes) // W
    counts[0] += torch.tensor(sizes) - counts.sum(0)
    rc = counts.view(-1).to(DEV)
    x, dh = rnd(A, H1), rnd(A, N, std=0.5)
    wg, wu = rnd(e, H1, N, std=H1 ** -0.5), rnd(e, H1, N, std=H1 ** -0.5)
    plan = binding.GatedPlan(W, e, A, H1, N, save=True)
    t = plan.run(x, rc, wg, wu)
    want = plan.backward(dh, t.permuteOut, rc, wg, wu, t.saved)
    assert binding.a2av_gmm_read_device_status(plan.workspace) == (0, 0)

    checks = binding.load_checks()
    checks.a2av_checks_slopes_short.argtypes = [ctypes.c_int32, ctypes.c_uint64]
    ordinary, binding._lib = binding._lib, checks
    try:
        checks.a2av_checks_slopes_short(1, 20_000_000)
        plan.backward(dh, t.permuteOut, rc, wg, wu, t.saved)
        name, bits = binding.a2av_gmm_read_device_status(plan.workspace)
        assert binding.STATUS_NAMES[name] == "A2AV_ERR_CUDA" and bits == TIMEOUT
    finally:
        checks.a2av_checks_slopes_short(0, 0)
        binding._lib = ordinary
    again = plan.backward(dh, t.permuteOut, rc, wg, wu, t.saved)
    assert binding.a2av_gmm_read_device_status(plan.workspace) == (0, 0)
    for p, q in zip(again, want):
        assert torch.equal(p.view(torch.int16), q.view(torch.int16))
