"""An expert layer's feed-forward part on one rank, from the library's operators.

Training (`ExpertBlock`), on the rows an exchange delivered (rank-major, with recvCounts):

    h = act(X Wg) * (X Wu)      a2av_gated_run        (permutes, both projections, activation, product)
    y = h Wd                    a2av_gmm_run          (one matrix per expert)

and backward from dy: a2av_gmm_backward, then a2av_gated_backward.  In front of the exchange,
binding.a2av_rms_norm makes the rows (y in the element type, or codes with scales) and the residual stream;
binding.a2av_rms_norm_backward takes the gradient back through both.

Serving in 8 bits (`MxExpertBlock`), on rows that arrive as the codes and scales a2av_rms_norm wrote:

    g|u = X [Wg | Wu]           a2av_gmm_mx_run
    h   = act(g) * u            a2av_glu_quant        (codes and scales out)
    y   = h Wd                  a2av_gmm_mx_run

Rows of h and y are expert-major.  Plans hold the workspaces, so one object serves every call of its shape.
"""

from __future__ import annotations

from typing import NamedTuple

import torch

from . import binding


def expert_counts(recvCounts: torch.Tensor, W: int, e: int) -> torch.Tensor:
    """Rows of each expert, int32 [e]: the counts of rows that are expert-major already (one source)."""
    return recvCounts if W == 1 else recvCounts.view(W, e).sum(0, dtype=torch.int32)


class BlockGrads(NamedTuple):
    dAtaOut: torch.Tensor  # [A, H], rank-major
    dGate: torch.Tensor    # [e, H, N]
    dUp: torch.Tensor      # [e, H, N]
    dDown: torch.Tensor    # [e, N, H]


class ExpertBlock:
    """y = (act(X Wg) * (X Wu)) Wd per expert, and its backward pass, for one shape: A rows of width H from W
    sources, e experts of inner width N."""

    def __init__(self, W, e, A, H, N, dtype=torch.bfloat16, act="silu", device=None):
        self.W, self.e = W, e
        self.gated = binding.GatedPlan(W, e, A, H, N, dtype, act, save=True, device=device)
        self.down = binding.Plan(1, e, A, N, H, dtype=dtype, device=self.gated.device)
        self.down_backward = binding.GmmBackwardPlan(1, e, A, N, H, dtype, device=self.gated.device)

    def forward(self, ataOut, recvCounts, gate, up, down):
        """(y [A, H], kept): kept is what backward() takes."""
        counts = expert_counts(recvCounts, self.W, self.e)
        g = self.gated.run(ataOut, recvCounts, gate, up)
        y, _, _ = self.down.run(g.h, counts, down)
        return y, (g, recvCounts, counts)

    def backward(self, dy, kept, gate, up, down) -> BlockGrads:
        g, recvCounts, counts = kept
        dh, dDown = self.down_backward.run(dy, g.h, counts, down)
        b = self.gated.backward(dh, g.permuteOut, recvCounts, gate, up, g.saved)
        return BlockGrads(b.dAtaOut, b.dGate, b.dUp, dDown)


class MxExpertBlock:
    """The same block in block-scaled FP8: codes and E8M0 scales in, y [A, H] bf16 out.  Weights as a2av_gmm_mx_run
    takes them: gate_up [e, 2N, H] (an expert's gate columns, then its up columns) and down [e, H, N]."""

    def __init__(self, W, e, A, H, N, act="silu", qtype="e4m3fn", device=None):
        self.W, self.e, self.act, self.qtype = W, e, act, qtype
        self.first = binding.MxPlan(W, e, A, H, 2 * N, qtype=qtype, device=device)
        self.down = binding.MxPlan(1, e, A, N, H, qtype=qtype, device=self.first.device)

    def forward(self, rows_q, rows_s, recvCounts, gate_up_q, gate_up_s, down_q, down_s):
        gu, _, _, _ = self.first.run(rows_q, rows_s, recvCounts, gate_up_q, gate_up_s)
        h = binding.a2av_glu_quant(gu, self.act, self.qtype, "mx")
        y, _, _, _ = self.down.run(h.codes, h.scales, expert_counts(recvCounts, self.W, self.e), down_q, down_s)
        return y
