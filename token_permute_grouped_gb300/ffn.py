"""An expert layer's feed-forward part on one rank, from the library's operators.

Training (`ExpertBlock`), on the rows an exchange delivered (rank-major, with recvCounts):

    h = act(X Wg) * (X Wu)      a2av_gated_run        (permutes, both projections, activation, product)
    y = h Wd                    a2av_gmm_run          (one matrix per expert)

and backward from dy: a2av_gmm_backward, then a2av_gated_backward.  In front of the exchange,
binding.a2av_rms_norm or binding.a2av_layer_norm makes the rows (y in the element type, or codes with scales) and the
residual stream; binding.a2av_rms_norm_backward or a2av_layer_norm_backward takes the gradient back through both.

Serving in 8 bits (`MxExpertBlock`), on rows that arrive as the codes and scales a2av_rms_norm wrote:

    g|u = X [Wg | Wu]           a2av_gmm_mx_run
    h   = act(g) * u            a2av_glu_quant        (codes and scales out)
    y   = h Wd                  a2av_gmm_mx_run

`G128ExpertBlock` is the same with a float32 scale per 128 codes (a2av_gmm_g128_run), as other checkpoints are kept.

A decode step of a few tokens on one GPU (`TokenLayer`), with all experts of the layer:

    n, s = norm(x + residual)   a2av_rms_norm or a2av_layer_norm (s: the residual stream)
    y    = s + experts(n)       a2av_moe_run          (router, choice, experts, weighted sum)

Rows of h and y are expert-major (TokenLayer's: the tokens').  Plans hold the workspaces, so one object serves every call
of its shape.  G128ExpertBlock, MxExpertBlock and TokenLayer serve; they have no gradients.
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


class G128ExpertBlock:
    """MxExpertBlock with float32 scales: one for 128 codes of a row, one for 128 columns x 128 codes of a weight.  Weights as
    a2av_gmm_g128_run takes them: gate_up [e, 2N, H] (an expert's gate columns, then its up columns) and down [e, H, N].
    H and N are multiples of 128; y [A, H] is of type dtype."""

    def __init__(self, W, e, A, H, N, dtype=torch.bfloat16, act="silu", qtype="e4m3fn", device=None):
        self.W, self.e, self.act, self.qtype = W, e, act, qtype
        self.first = binding.G128Plan(W, e, A, H, 2 * N, dtype, qtype, device=device)
        self.down = binding.G128Plan(1, e, A, N, H, dtype, qtype, device=self.first.device)

    def forward(self, rows_q, rows_s, recvCounts, gate_up_q, gate_up_s, down_q, down_s):
        gu = self.first.run(rows_q, rows_s, recvCounts, gate_up_q, gate_up_s)
        h = binding.a2av_glu_quant(gu, self.act, self.qtype, "group128")
        return self.down.run(h.codes, h.scales, expert_counts(recvCounts, self.W, self.e), down_q, down_s)


class TokenLayer:
    """A decode step's norm and expert layer for T tokens (up to 64): y = s + experts(norm(s)), s = x + residual (residual
    None: x): y is the residual stream behind the layer.  beta given: layer norm; else RMS norm."""

    def __init__(self, T, E, K, H, N, dtype=torch.bfloat16, act="silu", score="softmax", renormalise=True, scale=1.0,
                 router_dtype=None, eps=1e-6, device=None):
        self.eps = eps
        self.moe = binding.MoePlan(T, E, K, H, N, dtype, act, score, renormalise, scale, router_dtype, device)

    def forward(self, x, residual, gamma, router, gate, up, down, beta=None, bias=None) -> binding.MoeOut:
        if beta is None:
            n = binding.a2av_rms_norm(x, gamma, residual, self.eps, want_y=True)
        else:
            n = binding.a2av_layer_norm(x, gamma, beta, residual, self.eps, want_y=True)
        s = x if residual is None else n.h
        return self.moe.run(n.y, router, gate, up, down, bias=bias, residual=s)
