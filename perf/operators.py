"""Cases for timing and checking the operators around the grouped product: the RMS norm with the residual's
addition and 8-bit output, the gated feed-forward block over ragged experts, the gated activation with 8-bit
output, and the gradients of the norm, the gated block and the grouped product.

`run` computes a case either in its plain form (`own` false: elementary torch operations in float32, rounded once)
or through this repository's library (`own` true).  `exact` gives the same outputs in float64.

8-bit codes are returned as float8 tensors, E8M0 scales as float8_e8m0fnu: both compare as the values they stand
for.  INT8 codes are whole numbers whose last step may go either way at a tie of the float32 value, so the cases
use the two float8 formats only.
"""

import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16}
_F8 = {"e4m3fn": (torch.float8_e4m3fn, 8, 448.0), "e5m2": (torch.float8_e5m2, 15, 57344.0)}
EPS = 1e-6


# ------------------------------------------------------------------ cases


def listed():
    def norm(name, rows, H, dtype="bf16", qtype="e4m3fn", mode="mx", pad=0, want_y=False):
        return {"name": name, "op": "norm", "rows": rows, "H": H, "dtype": dtype, "qtype": qtype, "mode": mode,
                "pad": pad, "want_y": want_y}

    def gated(name, W, e, A, H1, N, dtype="bf16", act="silu", train=False, empty=0.0):
        return {"name": name, "op": "gated", "W": W, "e": e, "A": A, "H1": H1, "N": N, "dtype": dtype, "act": act,
                "train": train, "empty": empty}

    return [
        # One token of a decode step: the layer's input norm, codes for the dispatch.
        norm("norm_token", 1, 7168),
        # A prompt's tokens (eight ranks' 1536 rows) normed and quantised before the dispatch.
        norm("norm_prompt", 12288, 7168),
        # Rows of a wider buffer (row stride 2112), fp16, group-of-128 scales, the normed rows wanted as well.
        norm("norm_strided_odd", 4099, 2048, dtype="fp16", qtype="e5m2", mode="group128", pad=64, want_y=True),
        # The norm's gradient in a training step, the residual stream's gradient added in the same pass.
        {"name": "norm_grad", "op": "norm_grad", "rows": 16384, "H": 2048, "dtype": "bf16"},
        # Decode: eight rows, one from each rank, land on four local experts; latency and weight bytes count.
        gated("gated_token", 8, 4, 8, 4096, 1024),
        # Serving a prompt on one rank of 32 with skewed routing: no gradients, nothing kept.
        gated("gated_serve", 32, 8, 34502, 7168, 2048),
        # A training step's block, forward and backward, sixteen experts of about 4.1K rows.
        gated("gated_train", 16, 16, 65308, 2048, 1408, train=True),
        # fp16 training with odd sizes: widths that are no multiple of 64, a fifth of the segments empty.
        gated("gated_train_ragged", 8, 32, 5013, 1032, 328, dtype="fp16", act="gelu_tanh", train=True, empty=0.2),
        # Between the two block-scaled products of a served expert layer: gate and up columns to codes.
        {"name": "glu_prompt", "op": "glu", "rows": 34502, "N": 2048, "dtype": "bf16", "act": "silu",
         "qtype": "e4m3fn", "mode": "mx"},
        # A few rows, fp16, group-of-128 scales.
        {"name": "glu_few", "op": "glu", "rows": 37, "N": 1408, "dtype": "fp16", "act": "gelu_tanh",
         "qtype": "e5m2", "mode": "group128"},
        # The down projection's gradient in a training step, four experts.
        {"name": "gmm_grad", "op": "gmm_grad", "W": 8, "e": 4, "A": 16407, "H1": 1024, "N1": 4096, "dtype": "bf16",
         "empty": 0.0},
        # The smallest gradient: two ranks, two experts.
        {"name": "gmm_grad_small", "op": "gmm_grad", "W": 2, "e": 2, "A": 256, "H1": 256, "N1": 128,
         "dtype": "bf16", "empty": 0.0},
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], spread over its logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    v = min(max(v, lo), hi)
    return v + step if v == 3 * 1024 else v


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "gated", "gated", "gated", "glu", "gmm_grad"])
    dtype = rng.choice(["bf16", "fp16"])
    qtype, mode = rng.choice(["e4m3fn", "e5m2"]), rng.choice(["mx", "group128"])
    if op == "norm":
        return {"op": op, "rows": _spread(rng, 1, 12288), "H": _spread(rng, 256, 8192, 128), "dtype": dtype,
                "qtype": qtype, "mode": mode, "pad": rng.choice([0, 0, 8, 72]), "want_y": rng.random() < 0.3}
    if op == "norm_grad":
        return {"op": op, "rows": _spread(rng, 1, 16384), "H": _spread(rng, 256, 8192, 8), "dtype": dtype}
    if op == "glu":
        return {"op": op, "rows": _spread(rng, 1, 34502), "N": _spread(rng, 128, 2048, 128), "dtype": dtype,
                "act": rng.choice(["silu", "gelu_tanh"]), "qtype": qtype, "mode": mode}
    W, e = rng.choice([1, 2, 8, 16]), rng.choice([1, 2, 4, 7, 16])
    step = rng.choice([8, 64, 128])
    empty = rng.choice([0.0, 0.0, 0.2])
    A = _spread(rng, 1, 32768)
    if op == "gmm_grad":
        return {"op": op, "W": W, "e": e, "A": A, "H1": _spread(rng, 128, 2048, step), "N1": _spread(rng, 128, 4096, step),
                "dtype": dtype, "empty": empty}
    return {"op": op, "W": W, "e": e, "A": A, "H1": _spread(rng, 256, 4096, step), "N": _spread(rng, 128, 1408, step),
            "dtype": dtype, "act": rng.choice(["silu", "gelu_tanh"]), "train": A <= 16384 and rng.random() < 0.5,
            "empty": empty}


def work(case):
    op = case["op"]
    if op in ("norm", "glu"):
        cols = case["H"] if op == "norm" else case["N"]
        n = case["rows"] * cols
        scales = n // 32 if case["mode"] == "mx" else n // 128 * 4
        # norm: x, residual in; h, codes, scales (and y) out.  glu: gate, up in; codes, scales out.
        return {"bytes": n * (4 + 1) + scales + (n * 2 * (2 if case["want_y"] else 1) + cols * 2 if op == "norm" else 0),
                "flops": 8 * n}
    if op == "norm_grad":  # dy, dh, h in; dx out; rstd, gamma, dgamma
        n = case["rows"] * case["H"]
        return {"bytes": n * 8 + case["rows"] * 4 + case["H"] * 6, "flops": 12 * n}
    A, e, H1 = case["A"], case["e"], case["H1"]
    active = e * (1.0 - (1.0 - 1.0 / e) ** A) if A else 0.0  # experts that some row reaches, on average
    if op == "gmm_grad":
        N1 = case["N1"]
        # dY, the rows, the weights in; the rows' gradient and every expert's weight gradient out.
        return {"bytes": 2 * (A * N1 + A * H1 + active * H1 * N1 + A * H1 + e * H1 * N1), "flops": 4 * A * H1 * N1}
    N = case["N"]
    fwd = 2 * (A * H1 + active * 2 * H1 * N + A * N)
    if not case["train"]:
        return {"bytes": fwd, "flops": 4 * A * H1 * N}
    # backward on top: dh, the rows and the weights again; dX and the weights' gradients out.
    return {"bytes": fwd + 2 * (A * N + A * H1 + active * 2 * H1 * N + A * H1 + e * 2 * H1 * N),
            "flops": 12 * A * H1 * N}


# ------------------------------------------------------------------ inputs


def _counts(case, seed):
    """Rows of each (source rank, local expert) segment: normal logits with a bias for each expert, some segments
    forced empty; they sum to A."""
    rng = np.random.default_rng([seed, 11])
    W, e = case["W"], case["e"]
    p = np.exp(rng.normal(0.0, 0.15, (W, e)) + rng.normal(0.0, 0.4, e))
    gone = rng.permutation(W * e)[: int(case["empty"] * W * e)]
    p.reshape(-1)[gone] = 0.0
    return rng.multinomial(case["A"], p.reshape(-1) / p.sum()).astype(np.int32)


def prepare(case, seed):
    """The operands on the GPU, made from the seed; routing counts on the host and on the GPU, as a program that
    has just exchanged them has both."""
    dev, dt, op = torch.device("cuda"), _DT[case["dtype"]], case["op"]
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 1000003 + 17)

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return (torch.empty(*shape, dtype=torch.float32, device=dev).normal_(mean, std, generator=gen)).to(dtype)

    s = {"case": case}
    if op == "norm":
        rows, H, pad = case["rows"], case["H"], case["pad"]
        s["x"] = normal(rows, H + pad)[:, :H]
        s["residual"] = normal(rows, H, std=3.0)
        s["gamma"] = normal(H, std=0.1, mean=1.0)
    elif op == "norm_grad":
        rows, H = case["rows"], case["H"]
        s["h"] = normal(rows, H, std=3.0)
        s["gamma"] = normal(H, std=0.1, mean=1.0)
        s["dy"] = normal(rows, H, std=0.05)
        s["dh"] = normal(rows, H, std=0.05)
        s["rstd"] = torch.rsqrt(s["h"].float().square().mean(1) + EPS)
    elif op == "glu":
        s["gate_up"] = normal(case["rows"], 2 * case["N"], std=1.5)
    else:
        A, e, H1 = case["A"], case["e"], case["H1"]
        N = case["N"] if op == "gated" else case["N1"]
        c = _counts(case, seed)
        s["counts"] = c.tolist()
        s["recvCounts"] = torch.from_numpy(c).to(dev)
        s["x"] = normal(A, H1)
        if op == "gated":
            s["gate"] = normal(e, H1, N, std=H1 ** -0.5)
            s["up"] = normal(e, H1, N, std=H1 ** -0.5)
            if case["train"]:
                s["dout"] = normal(A, N, std=0.5)
        else:
            s["weight"] = normal(e, H1, N, std=H1 ** -0.5)
            s["dout"] = normal(A, N, std=0.5)
    return s


# ------------------------------------------------------------------ the plain form, in float32


def _act(g, name):
    if name == "silu":
        return g / (1.0 + torch.exp(-g))
    return 0.5 * g * (1.0 + torch.tanh(0.7978845608028654 * (g + 0.044715 * g * g * g)))


def _act_and_slope(g, name):
    if name == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    t = torch.tanh(0.7978845608028654 * (g + 0.044715 * g * g * g))
    slope = 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * 0.7978845608028654 * (1.0 + 3.0 * 0.044715 * g * g)
    return 0.5 * g * (1.0 + t), slope


def _quantise(y, qtype, mode):
    """float32 [rows, n] -> float8 codes, and E8M0 scales per 32 (mx) or float32 scales per 128 (group128)."""
    f8, emax, fmax = _F8[qtype]
    rows, n = y.shape
    b = y.view(rows, -1, 32 if mode == "mx" else 128)
    amax = b.abs().amax(2)
    if mode == "mx":
        exponent = (torch.frexp(amax)[1] - 1 - emax).clamp(-127, 127)
        exponent = torch.where(amax > 0, exponent, torch.full_like(exponent, -127))
        codes = torch.ldexp(b, -exponent[..., None]).clamp(-fmax, fmax).to(f8)
        return codes.view(rows, n), (exponent + 127).to(torch.uint8).view(torch.float8_e8m0fnu)
    amax = amax.clamp_min(2.0 ** -100)
    codes = (b * (fmax / amax)[..., None]).clamp(-fmax, fmax).to(f8)
    return codes.view(rows, n), amax / fmax


def _segments(x, counts, W, e):
    """Rank-major rows -> each expert's rows, sources in order."""
    parts = torch.split(x, counts)
    return [torch.cat([parts[w * e + j] for w in range(W)]) for j in range(e)]


def _to_arrival(groups, counts, W, e):
    """Each expert's rows -> rank-major rows."""
    parts = [torch.split(g, [counts[w * e + j] for w in range(W)]) for j, g in enumerate(groups)]
    return torch.cat([parts[j][w] for w in range(W) for j in range(e)])


def _expert_sizes(counts, W, e):
    return [sum(counts[w * e + j] for w in range(W)) for j in range(e)]


def _plain(s):
    case = s["case"]
    op, dt = case["op"], _DT[case["dtype"]]
    if op == "norm":
        t = s["x"].float() + s["residual"].float()
        y = t * torch.rsqrt((t * t).mean(1, keepdim=True) + EPS) * s["gamma"].float()
        codes, scales = _quantise(y, case["qtype"], case["mode"])
        return {"h": t.to(dt), "codes": codes, "scales": scales, **({"y": y.to(dt)} if case["want_y"] else {})}
    if op == "norm_grad":
        dy, n = s["dy"].float(), s["h"].float() * s["rstd"][:, None]
        a = dy * s["gamma"].float()
        dx = s["dh"].float() + s["rstd"][:, None] * (a - n * (a * n).mean(1, keepdim=True))
        return {"dx": dx.to(dt), "dgamma": (dy * n).sum(0)}
    if op == "glu":
        g, u = s["gate_up"].float().chunk(2, dim=1)
        codes, scales = _quantise(_act(g, case["act"]) * u, case["qtype"], case["mode"])
        return {"codes": codes, "scales": scales}
    W, e, counts = case["W"], case["e"], s["counts"]
    if op == "gmm_grad":  # the forward call's permuted rows: expert after expert
        sizes = _expert_sizes(counts, W, e)
        xs, w, dys = torch.split(s["x"].float(), sizes), s["weight"].float(), torch.split(s["dout"].float(), sizes)
        dx = _to_arrival([dy @ w[j].t() for j, dy in enumerate(dys)], counts, W, e)
        return {"dx": dx.to(dt), "dweight": torch.stack([x.t() @ dy for x, dy in zip(xs, dys)]).to(dt)}
    xs = _segments(s["x"].float(), counts, W, e)
    wg, wu = s["gate"].float(), s["up"].float()
    gs = [x @ wg[j] for j, x in enumerate(xs)]
    us = [x @ wu[j] for j, x in enumerate(xs)]
    if not case["train"]:
        return {"h": torch.cat([_act(g, case["act"]) * u for g, u in zip(gs, us)]).to(dt)}
    g, u, dh = torch.cat(gs), torch.cat(us), s["dout"].float()
    act, slope = _act_and_slope(g, case["act"])
    sizes = _expert_sizes(counts, W, e)
    dgs, dus = torch.split(dh * u * slope, sizes), torch.split(dh * act, sizes)
    dx = _to_arrival([a @ wg[j].t() + b @ wu[j].t() for j, (a, b) in enumerate(zip(dgs, dus))], counts, W, e)
    return {"h": (act * u).to(dt), "dx": dx.to(dt),
            "dgate": torch.stack([x.t() @ a for x, a in zip(xs, dgs)]).to(dt),
            "dup": torch.stack([x.t() @ b for x, b in zip(xs, dus)]).to(dt)}


# ------------------------------------------------------------------ the library's operators


def _own(s):
    from token_permute_grouped_gb300 import binding

    case = s["case"]
    op, dt = case["op"], _DT[case["dtype"]]
    if op == "norm":
        r = s["out"] = binding.a2av_rms_norm(s["x"], s["gamma"], s["residual"], EPS, case["qtype"], case["mode"],
                                             want_y=case["want_y"], out=s.get("out"))
        out = {"h": r.h, "codes": r.codes.view(_F8[case["qtype"]][0]),
               "scales": r.scales.view(torch.float8_e8m0fnu) if case["mode"] == "mx" else r.scales}
        if case["want_y"]:
            out["y"] = r.y
        return out
    if op == "norm_grad":
        dx, dgamma = binding.a2av_rms_norm_backward(s["dy"], s["h"], s["gamma"], s["rstd"], s["dh"])
        return {"dx": dx, "dgamma": dgamma}
    if op == "glu":
        r = s["out"] = binding.a2av_glu_quant(s["gate_up"], case["act"], case["qtype"], case["mode"],
                                              out=s.get("out"))
        return {"codes": r.codes.view(_F8[case["qtype"]][0]),
                "scales": r.scales.view(torch.float8_e8m0fnu) if case["mode"] == "mx" else r.scales}
    W, e, A, H1 = case["W"], case["e"], case["A"], case["H1"]
    if op == "gmm_grad":
        if "plan" not in s:
            s["plan"] = binding.GmmBackwardPlan(W, e, A, H1, case["N1"], dt)
        dx, dweight = s["plan"].run(s["dout"], s["x"], s["recvCounts"], s["weight"])
        return {"dx": dx, "dweight": dweight}
    if "plan" not in s:
        s["plan"] = binding.GatedPlan(W, e, A, H1, case["N"], dt, case["act"], save=case["train"])
    plan = s["plan"]
    if not case["train"]:
        h = s["out"] = plan.run(s["x"], s["recvCounts"], s["gate"], s["up"], h=s.get("out")).h
        return {"h": h}
    f = plan.run(s["x"], s["recvCounts"], s["gate"], s["up"])
    b = plan.backward(s["dout"], f.permuteOut, s["recvCounts"], s["gate"], s["up"], f.saved)
    return {"h": f.h, "dx": b.dAtaOut, "dgate": b.dGate, "dup": b.dUp}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ the definition, in float64


def _exact_codes(y, qtype, mode):
    """What the codes and scales stand for, unrounded: y over its block's scale (saturating), and the scale."""
    _, emax, fmax = _F8[qtype]
    block = 32 if mode == "mx" else 128
    blocks = y.unflatten(1, (y.shape[1] // block, block))
    top = blocks.abs().max(2).values
    if mode == "mx":
        scale = torch.exp2(torch.floor(torch.log2(top)).clamp(-127 + emax, 127 + emax) - emax)
    else:
        scale = torch.maximum(top, torch.full_like(top, 2.0 ** -100)) / fmax
    codes = torch.clamp(blocks / scale.unsqueeze(2), min=-fmax, max=fmax).flatten(1)
    return codes, scale


def _exact_gated(x, wg, wu, act):
    g = x @ wg
    a = g * torch.sigmoid(g) if act == "silu" else torch.nn.functional.gelu(g, approximate="tanh")
    return a * (x @ wu)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor) and v.is_floating_point()}
    if op == "norm":
        h = d["x"] + d["residual"]
        y = h / torch.sqrt(h.pow(2).sum(1, keepdim=True) / case["H"] + EPS) * d["gamma"]
        codes, scales = _exact_codes(y, case["qtype"], case["mode"])
        return {"h": h, "codes": codes, "scales": scales, **({"y": y} if case["want_y"] else {})}
    if op == "norm_grad":
        # With rstd given, the row's gradient is the formula's; written over the dot product of dy * gamma and h.
        r, w = d["rstd"].unsqueeze(1), d["dy"] * d["gamma"]
        dot = (w * d["h"]).sum(1, keepdim=True)
        return {"dx": d["dh"] + r * w - r.pow(3) * dot / case["H"] * d["h"],
                "dgamma": torch.einsum("rh,rh,r->h", d["dy"], d["h"], d["rstd"])}
    if op == "glu":
        g, u = d["gate_up"][:, :case["N"]], d["gate_up"][:, case["N"]:]
        a = g * torch.sigmoid(g) if case["act"] == "silu" else torch.nn.functional.gelu(g, approximate="tanh")
        codes, scales = _exact_codes(a * u, case["qtype"], case["mode"])
        return {"codes": codes, "scales": scales}
    # Each arrival row's expert; an expert's rows keep their order of arrival.  (The grouped product's gradient has its
    # rows in expert order already.)
    e, dev = case["e"], d["x"].device
    owner = torch.repeat_interleave(torch.arange(case["W"] * e, device=dev) % e, s["recvCounts"].long())
    x, at = d["x"], 0
    dx = torch.zeros_like(x)
    hs, dws = [], []
    for j in range(e):
        rows = torch.nonzero(owner == j).flatten()
        n = rows.numel()
        xj = (x[at:at + n] if op == "gmm_grad" else x[rows]).requires_grad_(True)
        if op == "gmm_grad":
            wj = [d["weight"][j].requires_grad_(True)]
            hj = xj @ wj[0]
        else:
            wj = [d["gate"][j].requires_grad_(True), d["up"][j].requires_grad_(True)]
            hj = _exact_gated(xj, wj[0], wj[1], case["act"])
        if "dout" in d:
            grads = torch.autograd.grad(hj, [xj] + wj, d["dout"][at:at + n])
            dx[rows] = grads[0]
            dws.append(grads[1:])
        hs.append(hj.detach())
        at += n
    if op == "gmm_grad":
        return {"dx": dx, "dweight": torch.stack([g[0] for g in dws])}
    if not case["train"]:
        return {"h": torch.cat(hs)}
    return {"h": torch.cat(hs), "dx": dx, "dgate": torch.stack([g[0] for g in dws]),
            "dup": torch.stack([g[1] for g in dws])}
