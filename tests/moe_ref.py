"""Plain float64 form of the expert layer for a few tokens, and the bounds on the library's errors (see ffn_ref.py for u,
step, CHAIN and the products' slack).

A logit is a sum of fp32 sums of at most 2 H / 256 + 2 products a thread (a vector of 8 at a time, two halves), joined with
their rounding errors: within (H / 128 + 8) 2^-24 of the sum of magnitudes.  A score moves by at most twice a logit's error,
and its own exponentials, sums and quotients are within CHAIN.  A gated value goes on as two summands of the element type:
the first within 2 u of it (toward zero), the second rounds the rest, u of it and at most a step."""

import torch

import ffn_ref as R

GAP = 2.0 ** -16  # keys nearer than this may be chosen in either order


def route(x, router, K, score="softmax", renormalise=True, scale=1.0, bias=None):
    """experts [T, K], weights [T, K], the bound on the weights' relative errors [T, K], and whether a token's choice and
    its order are beyond doubt [T]."""
    x, router = x.double(), router.double()
    logits = x @ router.t()
    el = ((x.shape[1] / 128 + 8) * 2.0 ** -24 * (x.abs() @ router.abs().t())).amax(1, keepdim=True)
    p = torch.softmax(logits, 1) if score == "softmax" else torch.sigmoid(logits)
    key = logits if bias is None else p + bias.double()
    order = torch.sort(key, dim=1, descending=True, stable=True)
    experts = order.indices[:, :K]
    gaps = (order.values[:, :-1] - order.values[:, 1:])[:, :K] if key.shape[1] > 1 else key.new_ones(len(key), 1)
    w = p.gather(1, experts)
    if renormalise:
        w = w / w.sum(1, keepdim=True)
    return experts, w * scale, (4 * el + R.CHAIN).expand_as(w), (gaps > GAP + 4 * el).all(1)


def values(x, experts, weights, ew, gate, up, down, act, residual, dtype):
    """y and the bound on its error before its rounding, for these choices and weights."""
    x = x.double()
    T, K = experts.shape
    H, N = gate.shape[1:]
    y = residual.double().clone() if residual is not None else torch.zeros_like(x)
    err = 2.0 ** -23 * y.abs()
    u, step = R.U[dtype], R.STEP[dtype]
    for t in range(T):
        for k in range(K):
            e = int(experts[t, k])
            wg, wu, wd = gate[e].double(), up[e].double(), down[e].double()
            g, v = x[t] @ wg, x[t] @ wu
            slack = (H + 8) * 2.0 ** -23
            eg, ev = slack * (x[t].abs() @ wg.abs()), slack * (x[t].abs() @ wu.abs())
            a = R.act(g, act)
            h = a * v
            eh = 1.13 * eg * (v.abs() + ev) + a.abs() * ev + R.CHAIN * h.abs() + 2 * u * u * h.abs() + step
            d = h @ wd
            ed = eh @ wd.abs() + (2 * N + 8) * 2.0 ** -23 * ((h.abs() + eh) @ wd.abs())
            w = float(weights[t, k])
            y[t] += w * d
            err[t] += abs(w) * (1 + float(ew[t, k])) * ed + abs(w) * float(ew[t, k]) * d.abs() \
                + (K + 2) * 2.0 ** -23 * (abs(w) * d.abs() + y[t].abs())
    return y, err
