"""Plain float64 form of the grouped product of codes with a float32 scale per 128, a quantiser of weights for the tests,
and the bound on the library's error.

A product of two codes is exact in fp32.  A block's 128 terms are added by the tensor cores (one rounding or truncation a
term, within (128 + 8) 2^-23 of the sum of magnitudes), its sum is scaled by a rounded product and added by one fused
operation a block, K / 128 of them: (K / 128 + 1) 2^-23 more."""

import torch

import ffn_ref as R


def values(codes, scales, qtype, columns=1):
    """Codes [..., n, K] and their scales, one for `columns` rows x 128 codes, in float64."""
    v = codes.cpu().view(R.F8[qtype][0]).double()
    n, K = v.shape[-2:]
    s = scales.cpu().double().repeat_interleave(columns, -2)[..., :n, :].repeat_interleave(128, -1)
    return v * s


def product(xq, xs, counts, W, e, wq, ws, qtype):
    """y [A, N] in float64, expert-major, and the bound on its error before the output's rounding."""
    idx, sizes = R.arrival_index(counts, W, e)
    x, w = values(xq, xs, qtype)[idx], values(wq, ws, qtype, 128)
    K = x.shape[1]
    y = torch.cat(R.per_expert(lambda j, r: r @ w[j].t(), sizes, x))
    mag = torch.cat(R.per_expert(lambda j, r: r.abs() @ w[j].abs().t(), sizes, x))
    return y, (136 + K // 128 + 1) * 2.0 ** -23 * mag


def quantise(v, qtype, rows):
    """Codes (uint8) and float32 scales of v [..., n, K], one for `rows` rows x 128 values."""
    f8, _, top, _, _ = R.F8[qtype]
    n, K = v.shape[-2:]
    b = torch.nn.functional.pad(v.float(), (0, 0, 0, -n % rows)).unflatten(-2, (-1, rows)).unflatten(-1, (-1, 128))
    s = b.abs().amax((-3, -1)).clamp_min(2.0 ** -100) / top
    q = (b / s[..., :, None, :, None]).clamp(-top, top).to(f8)
    return q.flatten(-2, -1).flatten(-3, -2)[..., :n, :].contiguous().view(torch.uint8), s
