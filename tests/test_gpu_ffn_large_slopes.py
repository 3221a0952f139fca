"""The gated block's backward pass for large finite pre-activations, where the activations' slopes are 0 or 1 and their
parts overflow, against float64 (on the GPU).  Bounds: tests/ffn_ref.py."""

import pytest
import torch

import ffn_ref as R
from token_permute_grouped_gb300 import binding, build

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    build.build()


@pytest.mark.parametrize("A", [20, 70])
@pytest.mark.parametrize("name", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
def test_large_pre_activations(A, name, dt):
    H1, N = 64, 96
    g = torch.Generator().manual_seed(1)
    rnd = lambda *s, std=1.0: torch.randn(*s, generator=g) * std
    x, wg, wu, dh = rnd(A, H1).to(dt), rnd(1, H1, N).to(dt), rnd(1, H1, N).to(dt), rnd(A, N).to(dt)
    G, U = rnd(A, N, std=2.0), rnd(A, N)
    big = torch.tensor([10.0, 30.0, 100.0, 1e6, 1e12, 1.3e13, 1e14, 1e18, 1e20, 1e30, 3e38])
    G[3, :22] = torch.cat([big, -big])
    G[A - 1, 40:62] = torch.cat([-big, big])
    f = {"xe": x.double(), "sizes": [A], "idx": torch.arange(A), "G": G.double(), "U": U.double(),
         "eg": torch.zeros(A, N).double(), "eu": torch.zeros(A, N).double()}
    (dx, ex), ((dg, eg), (du, eu)) = R.gated_backward(f, dh, wg, wu, name, dt)
    assert bool(torch.isfinite(dg).all())
    plan = binding.GatedPlan(1, 1, A, H1, N, dt, name, save=True)
    rc = torch.tensor([A], dtype=torch.int32, device="cuda")
    b = plan.backward(dh.cuda(), x.cuda(), rc, wg.cuda(), wu.cuda(), torch.stack([G, U]).cuda())
    R.assert_rounded(b.dGate, dg, eg, "dGate")
    small = torch.ones(A, dtype=torch.bool)
    small[[3, A - 1]] = False  # (their other factor, the activation itself, passes the type's range)
    R.assert_rounded(b.dAtaOut[small.cuda()], dx[small], ex[small], "dAtaOut")
    cols = G.abs().amax(0) < 100
    R.assert_rounded(b.dUp[:, :, cols.cuda()], du[:, :, cols], eu[:, :, cols], "dUp")
