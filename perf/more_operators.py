"""Cases for timing and checking the layer norm with the residual's addition and 8-bit output, its gradient, the
grouped product of 8-bit rows with a float32 scale per 128, and the whole expert layer for a few tokens.

`run` computes a case either in its plain form (`own` false: elementary torch operations in float32, the router's
choice in float64, rounded once) or through this repository's library (`own` true).  `exact` gives the same outputs in
float64.

8-bit codes are returned as float8 tensors, E8M0 scales as float8_e8m0fnu: both compare as the values they stand for.
"""

import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_F8 = {"e4m3fn": (torch.float8_e4m3fn, 8, 448.0), "e5m2": (torch.float8_e5m2, 15, 57344.0)}
EPS = 1e-5


# ------------------------------------------------------------------ cases


def listed():
    def norm(name, rows, H, dtype="bf16", qtype=None, mode="mx", pad=0, want_y=False, stats=False):
        return {"name": name, "op": "norm", "rows": rows, "H": H, "dtype": dtype, "qtype": qtype, "mode": mode,
                "pad": pad, "want_y": want_y, "stats": stats}

    def gmm(name, W, e, A, H1, N1, dtype="bf16", qtype="e4m3fn", empty=0.0):
        return {"name": name, "op": "gmm", "W": W, "e": e, "A": A, "H1": H1, "N1": N1, "dtype": dtype, "qtype": qtype,
                "empty": empty}

    def moe(name, T, E, K, H, N, dtype="bf16", act="silu", score="softmax", renormalise=True, scale=1.0, bias=False,
            router="same", residual=True):
        return {"name": name, "op": "moe", "T": T, "E": E, "K": K, "H": H, "N": N, "dtype": dtype, "act": act,
                "score": score, "renormalise": renormalise, "scale": scale, "bias": bias, "router": router,
                "residual": residual}

    return [
        # One token of a decode step: the layer's input norm, codes for the dispatch.
        norm("norm_token", 1, 7168, qtype="e5m2", mode="mx"),
        # A prompt's tokens (eight ranks' 1536 rows) normed and quantised before the dispatch.
        norm("norm_prompt", 12288, 7168, qtype="e4m3fn", mode="group128"),
        # Training on rows of a wider buffer, fp16, a width that is no multiple of 64: the normed rows, the residual
        # stream and both statistics for the backward pass.
        norm("norm_train_odd", 4099, 2056, dtype="fp16", pad=64, want_y=True, stats=True),
        # The norm's gradient in a training step, the residual stream's gradient added in the same pass.
        {"name": "norm_grad", "op": "norm_grad", "rows": 16384, "H": 2048, "dtype": "bf16"},
        # The gradient of a few rows (a short sequence of a fine-tuning step).
        {"name": "norm_grad_few", "op": "norm_grad", "rows": 61, "H": 4096, "dtype": "fp16"},
        # Decode: eight rows, one from each rank, land on four local experts; latency and weight bytes count.
        gmm("gmm_token", 8, 4, 8, 4096, 2048),
        # Serving a prompt on one rank of 32 with skewed routing: gate and up columns in one product.
        gmm("gmm_prompt", 32, 8, 34502, 7168, 4096),
        # Odd sizes: widths that are no multiple of 64 or 256, E5M2, fp16 out, a fifth of the segments empty.
        gmm("gmm_ragged", 8, 32, 5013, 1152, 328, dtype="fp16", qtype="e5m2", empty=0.2),
        # A batch of decode steps of many users: about a hundred rows an expert.
        gmm("gmm_batch", 16, 16, 1634, 2048, 2816),
        # One token through a layer of 32 experts.
        moe("moe_token", 1, 32, 4, 4096, 1024),
        # A few sequences decoded together over 256 experts, fp16, sigmoid scores with a selection bias, a router kept
        # in float32.
        moe("moe_few", 5, 256, 8, 4096, 1536, dtype="fp16", score="sigmoid", scale=2.5, bias=True, router="fp32"),
        # The largest batch: nearly every expert's weights are read.
        moe("moe_batch", 64, 256, 8, 2048, 1408, act="gelu_tanh", renormalise=False),
    ]


def _spread(rng, lo, hi, step=1):
    """A multiple of step in [lo, hi], spread over its logarithm."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step
    return min(max(v, lo), hi)


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_grad", "gmm", "gmm", "gmm", "moe", "moe", "moe"])
    dtype = rng.choice(["bf16", "fp16"])
    if op == "norm":
        qtype = rng.choice([None, "e4m3fn", "e5m2"])
        return {"op": op, "rows": _spread(rng, 1, 12288), "H": _spread(rng, 256, 7168, 128 if qtype else 8),
                "dtype": dtype, "qtype": qtype, "mode": rng.choice(["mx", "group128"]), "pad": rng.choice([0, 0, 8, 72]),
                "want_y": qtype is None or rng.random() < 0.3, "stats": rng.random() < 0.5}
    if op == "norm_grad":
        return {"op": op, "rows": _spread(rng, 1, 16384), "H": _spread(rng, 256, 7168, 8), "dtype": dtype}
    if op == "gmm":
        return {"op": op, "W": rng.choice([1, 2, 8, 16]), "e": rng.choice([1, 2, 4, 7, 16]), "A": _spread(rng, 1, 32768),
                "H1": _spread(rng, 128, 4096, 128), "N1": _spread(rng, 128, 4096, rng.choice([8, 64, 128])),
                "dtype": dtype, "qtype": rng.choice(["e4m3fn", "e5m2"]), "empty": rng.choice([0.0, 0.0, 0.2])}
    step = rng.choice([8, 64, 128])
    H, N = _spread(rng, 256, 4096, step), _spread(rng, 128, 1536, step)
    E = _spread(rng, 4, 256)
    while E * H * N > 256 * 2048 * 1408:
        E = E * 2 // 3
    return {"op": op, "T": _spread(rng, 1, 64), "E": E, "K": rng.randint(1, min(8, E)), "H": H, "N": N, "dtype": dtype,
            "act": rng.choice(["silu", "gelu_tanh"]), "score": rng.choice(["softmax", "sigmoid"]),
            "renormalise": rng.random() < 0.5, "scale": rng.choice([1.0, 1.0, 2.5]), "bias": rng.random() < 0.3,
            "router": rng.choice(["same", "same", "fp32"]), "residual": rng.random() < 0.5}


def work(case):
    op = case["op"]
    if op == "norm":  # x, residual, gamma, beta in; h, y, codes and scales, statistics out
        n, bytes_ = case["rows"] * case["H"], case["H"] * 4
        bytes_ += n * 6 + (n * 2 if case["want_y"] else 0) + (case["rows"] * 8 if case["stats"] else 0)
        if case["qtype"]:
            bytes_ += n + (n // 32 if case["mode"] == "mx" else n // 128 * 4)
        return {"bytes": bytes_, "flops": 10 * n}
    if op == "norm_grad":  # dy, dh, h in; dx out; the statistics, gamma, dgamma, dbeta
        n = case["rows"] * case["H"]
        return {"bytes": n * 8 + case["rows"] * 8 + case["H"] * 10, "flops": 15 * n}
    if op == "gmm":
        A, e, H1, N1 = case["A"], case["e"], case["H1"], case["N1"]
        active = e * (1.0 - (1.0 - 1.0 / e) ** A)  # experts that some row reaches, on average
        return {"bytes": A * (H1 + H1 // 32) + active * H1 * N1 * (1.0 + 4.0 / 16384) + 2 * A * N1,
                "flops": 2 * A * H1 * N1}
    T, E, K, H, N = (case[k] for k in ("T", "E", "K", "H", "N"))
    active = E * (1.0 - (1.0 - K / E) ** T)
    return {"bytes": active * 6 * H * N + E * H * (4 if case["router"] == "fp32" else 2) + (3 if case["residual"] else 2)
            * 2 * T * H + 8 * T * K, "flops": 6 * T * K * H * N + 2 * T * E * H}


# ------------------------------------------------------------------ inputs


def _counts(case, seed):
    """Rows of each (source rank, local expert) segment: normal logits with a bias for each expert, some segments
    forced empty; they sum to A."""
    rng = np.random.default_rng([seed, 13])
    W, e = case["W"], case["e"]
    p = np.exp(rng.normal(0.0, 0.15, (W, e)) + rng.normal(0.0, 0.4, e))
    p.reshape(-1)[rng.permutation(W * e)[: int(case["empty"] * W * e)]] = 0.0
    return rng.multinomial(case["A"], p.reshape(-1) / p.sum()).astype(np.int32)


def prepare(case, seed):
    """The operands on the GPU, made from the seed; routing counts on the host and on the GPU, as a program that has
    just exchanged them has both."""
    dev, dt, op = torch.device("cuda"), _DT[case["dtype"]], case["op"]
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 1000003 + 29)

    def normal(*shape, std=1.0, mean=0.0, dtype=dt):
        return torch.empty(*shape, dtype=torch.float32, device=dev).normal_(mean, std, generator=gen).to(dtype)

    s = {"case": case}
    if op == "norm":
        rows, H = case["rows"], case["H"]
        s["x"] = normal(rows, H + case["pad"], mean=0.25)[:, :H]
        s["residual"] = normal(rows, H, std=3.0, mean=0.5)
        s["gamma"], s["beta"] = normal(H, std=0.1, mean=1.0), normal(H, std=0.1)
    elif op == "norm_grad":
        rows, H = case["rows"], case["H"]
        s["h"] = normal(rows, H, std=3.0, mean=0.75)
        s["gamma"] = normal(H, std=0.1, mean=1.0)
        s["dy"], s["dh"] = normal(rows, H, std=0.05), normal(rows, H, std=0.05)
        h = s["h"].double()
        s["mean"] = h.mean(1).float()
        s["rstd"] = torch.rsqrt(h.var(1, unbiased=False) + EPS).float()
    elif op == "gmm":
        A, e, H1, N1 = case["A"], case["e"], case["H1"], case["N1"]
        c = _counts(case, seed)
        s["counts"] = c.tolist()
        s["recvCounts"] = torch.from_numpy(c).to(dev)
        # Rows and weights as a quantiser of blocks leaves them; columns differ in size, so the blocks' scales do too.
        size = torch.exp(normal(H1, dtype=torch.float32))
        x = normal(A, H1, dtype=torch.float32) * size
        s["codes"], s["scales"] = _block_codes(x, case["qtype"], 1)
        codes, scales = [], []
        for _ in range(e):
            q, sc = _block_codes(normal(N1, H1, std=H1 ** -0.5, dtype=torch.float32), case["qtype"], 128)
            codes.append(q)
            scales.append(sc)
        s["weight_codes"], s["weight_scales"] = torch.stack(codes), torch.stack(scales)
    else:
        T, E, H, N = case["T"], case["E"], case["H"], case["N"]
        s["x"] = normal(T, H)
        s["router"] = normal(E, H, std=1.5 * H ** -0.5, dtype=dt if case["router"] == "same" else torch.float32)
        if case["bias"]:
            s["bias"] = normal(E, std=0.1, dtype=torch.float32)
        if case["residual"]:
            s["residual"] = normal(T, H)
        for name, shape in (("gate", (H, N)), ("up", (H, N)), ("down", (N, H))):
            w = torch.empty(E, *shape, dtype=dt, device=dev)
            for j in range(E):
                w[j] = normal(*shape, std=shape[0] ** -0.5)
            s[name] = w
    return s


def _block_codes(v, qtype, rows):
    """float32 [n, K] -> uint8 codes [n, K] and a float32 scale for each block of `rows` x 128: largest magnitude over
    the format's largest value."""
    f8, _, fmax = _F8[qtype]
    n, K = v.shape
    pad = -n % rows
    b = torch.nn.functional.pad(v, (0, 0, 0, pad)).view((n + pad) // rows, rows, K // 128, 128)
    scales = b.abs().amax((1, 3)).clamp_min(2.0 ** -100) / fmax
    codes = (b / scales[:, None, :, None]).clamp(-fmax, fmax).to(f8)
    return codes.view(n + pad, K)[:n].contiguous().view(torch.uint8), scales


# ------------------------------------------------------------------ the plain form, in float32


def _act(g, name):
    if name == "silu":
        return g / (1.0 + torch.exp(-g))
    return 0.5 * g * (1.0 + torch.tanh(0.7978845608028654 * (g + 0.044715 * g * g * g)))


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


def _choose(logits, case, bias):
    """Router logits in float64 -> the chosen experts [T, K], largest first, and their weights in float32."""
    if case["score"] == "softmax":
        p = torch.exp(logits - logits.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-logits))
    key = p if bias is None else p + bias.double()
    experts = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :case["K"]]
    w = p.gather(1, experts)
    if case["renormalise"]:
        w = w / w.sum(1, keepdim=True)
    return experts.to(torch.int32), (w * case["scale"]).float()


def _plain(s):
    case = s["case"]
    op, dt = case["op"], _DT[case["dtype"]]
    if op == "norm":
        t = s["x"].float() + s["residual"].float()
        mean = t.mean(1, keepdim=True)
        d = t - mean
        rstd = torch.rsqrt((d * d).mean(1, keepdim=True) + EPS)
        y = d * rstd * s["gamma"].float() + s["beta"].float()
        out = {"h": t.to(dt)}
        if case["want_y"]:
            out["y"] = y.to(dt)
        if case["qtype"]:
            out["codes"], out["scales"] = _quantise(y, case["qtype"], case["mode"])
        if case["stats"]:
            out["mean"], out["rstd"] = mean[:, 0], rstd[:, 0]
        return out
    if op == "norm_grad":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        n = (s["h"].float() - s["mean"][:, None]) * rstd
        a = dy * s["gamma"].float()
        dx = s["dh"].float() + rstd * (a - a.mean(1, keepdim=True) - n * (a * n).mean(1, keepdim=True))
        return {"dx": dx.to(dt), "dgamma": (dy * n).sum(0), "dbeta": dy.sum(0)}
    if op == "gmm":
        W, e, counts, f8 = case["W"], case["e"], s["counts"], _F8[case["qtype"]][0]
        x = s["codes"].view(f8).float() * s["scales"].repeat_interleave(128, 1)
        parts, ys = torch.split(x, counts), []
        for j in range(e):
            w = s["weight_codes"][j].view(f8).float()
            w = w * s["weight_scales"][j].repeat_interleave(128, 0)[:case["N1"]].repeat_interleave(128, 1)
            ys.append(torch.cat([parts[r * e + j] for r in range(W)]) @ w.t())
        return {"y": torch.cat(ys).to(dt)}
    experts, weights = _choose(s["x"].double() @ s["router"].double().t(), case, s.get("bias"))
    x = s["x"].float()
    share = torch.zeros(case["T"], case["E"], device=x.device).scatter_(1, experts.long(), weights)
    y = s["residual"].float() if case["residual"] else torch.zeros_like(x)
    for j in range(case["E"]):
        h = _act(x @ s["gate"][j].float(), case["act"]) * (x @ s["up"][j].float())
        y = y + share[:, j:j + 1] * (h @ s["down"][j].float())
    return {"y": y.to(dt), "experts": experts, "weights": weights}


# ------------------------------------------------------------------ the library's operators


def _own(s):
    from token_permute_grouped_gb300 import binding

    case = s["case"]
    op, dt = case["op"], _DT[case["dtype"]]
    if op == "norm":
        r = s["out"] = binding.a2av_layer_norm(s["x"], s["gamma"], s["beta"], s["residual"], EPS, case["qtype"],
                                               case["mode"], want_y=case["want_y"], want_stats=case["stats"],
                                               out=s.get("out"))
        out = {"h": r.h}
        if case["want_y"]:
            out["y"] = r.y
        if case["qtype"]:
            out["codes"] = r.codes.view(_F8[case["qtype"]][0])
            out["scales"] = r.scales.view(torch.float8_e8m0fnu) if case["mode"] == "mx" else r.scales
        if case["stats"]:
            out["mean"], out["rstd"] = r.mean, r.rstd
        return out
    if op == "norm_grad":
        dx, dgamma, dbeta = binding.a2av_layer_norm_backward(s["dy"], s["h"], s["gamma"], s["mean"], s["rstd"], s["dh"])
        return {"dx": dx, "dgamma": dgamma, "dbeta": dbeta}
    if op == "gmm":
        if "plan" not in s:
            s["plan"] = binding.G128Plan(case["W"], case["e"], case["A"], case["H1"], case["N1"], dt, case["qtype"])
        y = s["y"] = s["plan"].run(s["codes"], s["scales"], s["recvCounts"], s["weight_codes"], s["weight_scales"],
                                   gmmY=s.get("y"))
        return {"y": y}
    if "plan" not in s:
        s["plan"] = binding.MoePlan(case["T"], case["E"], case["K"], case["H"], case["N"], dt, case["act"],
                                    case["score"], case["renormalise"], case["scale"],
                                    dt if case["router"] == "same" else torch.float32)
    r = s["out"] = s["plan"].run(s["x"], s["router"], s["gate"], s["up"], s["down"], bias=s.get("bias"),
                                 residual=s.get("residual"), out=s.get("out"))
    return {"y": r.y, "experts": r.experts, "weights": r.weights}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------------ the definition, in float64


def _exact_codes(y, qtype, mode):
    """The codes' values, y over its block's scale rounded to the format's grid (nearest even, saturating), and the
    scale."""
    _, emax, fmax = _F8[qtype]
    bits, low = (3, -6) if qtype == "e4m3fn" else (2, -14)  # of the fraction; exponent of the smallest normal value
    block = 32 if mode == "mx" else 128
    blocks = y.unflatten(1, (y.shape[1] // block, block))
    top = blocks.abs().max(2).values
    if mode == "mx":
        scale = torch.exp2(torch.floor(torch.log2(top)).clamp(-127 + emax, 127 + emax) - emax)
    else:
        scale = torch.maximum(top, torch.full_like(top, 2.0 ** -100)) / fmax
    v = torch.clamp(blocks / scale.unsqueeze(2), min=-fmax, max=fmax).flatten(1)
    step = torch.exp2(torch.floor(torch.log2(v.abs())).clamp_min(low) - bits)
    return torch.round(v / step) * step, scale


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        h = s["x"].double() + s["residual"].double()
        mean, H = h.sum(1) / case["H"], case["H"]
        # The second moment about the mean, from the sums of the values less their first.
        rel = h - h[:, :1]
        var = (rel.pow(2).sum(1) - rel.sum(1).pow(2) / H) / H
        rstd = 1.0 / torch.sqrt(var + EPS)
        y = torch.addcmul(s["beta"].double(), (h - mean.unsqueeze(1)) * rstd.unsqueeze(1), s["gamma"].double())
        out = {"h": h}
        if case["want_y"]:
            out["y"] = y
        if case["qtype"]:
            out["codes"], out["scales"] = _exact_codes(y, case["qtype"], case["mode"])
        if case["stats"]:
            out["mean"], out["rstd"] = mean, rstd
        return out
    if op == "norm_grad":
        # With the statistics given, the row's gradient is the formula's; written over the sums of w and of w (h - mean).
        r, w = s["rstd"].double().unsqueeze(1), s["dy"].double() * s["gamma"].double()
        c = s["h"].double() - s["mean"].double().unsqueeze(1)
        total, dot = w.sum(1, keepdim=True), (w * c).sum(1, keepdim=True)
        return {"dx": s["dh"].double() + r * w - r * total / case["H"] - r.pow(3) * c * dot / case["H"],
                "dgamma": torch.einsum("rh,rh,r->h", s["dy"].double(), c, r[:, 0]),
                "dbeta": torch.einsum("rh->h", s["dy"].double())}
    if op == "gmm":
        # Each arrival row's expert; an expert's rows keep their order of arrival.
        f8, e, K = _F8[case["qtype"]][0], case["e"], case["H1"]
        dev = s["codes"].device
        owner = torch.repeat_interleave(torch.arange(case["W"] * e, device=dev) % e, s["recvCounts"].long())
        ys = []
        for j in range(e):
            rows = torch.nonzero(owner == j).flatten()
            x = s["codes"][rows].view(f8).double().unflatten(1, (K // 128, 128))
            x = (x * s["scales"][rows].double().unsqueeze(2)).flatten(1)
            w = s["weight_codes"][j].view(f8).double()
            for b in range(s["weight_scales"].shape[1]):
                block = w[128 * b:128 * b + 128].unflatten(1, (K // 128, 128))
                block *= s["weight_scales"][j, b].double()[:, None]
            ys.append(torch.einsum("ik,nk->in", x, w))
        return {"y": torch.cat(ys)}
    T, K = case["T"], case["K"]
    x = s["x"].double()
    logits = torch.einsum("th,eh->te", x, s["router"].double())
    p = torch.softmax(logits, 1) if case["score"] == "softmax" else torch.sigmoid(logits)
    key = p + s["bias"].double() if case["bias"] else p.clone()
    experts = torch.empty(T, K, dtype=torch.int32, device=x.device)
    for k in range(K):  # the largest that is left; argmax of a row's maximum's first place
        top = (key == key.max(1, keepdim=True).values).to(torch.uint8).argmax(1)
        experts[:, k] = top
        key[torch.arange(T, device=x.device), top] = -math.inf
    w = torch.gather(p, 1, experts.long())
    w = w * (case["scale"] / w.sum(1, keepdim=True)) if case["renormalise"] else w * case["scale"]
    y = s["residual"].double() if case["residual"] else torch.zeros_like(x)
    for j in experts.unique().tolist():
        t, k = torch.nonzero(experts == j, as_tuple=True)
        g = x[t] @ s["gate"][j].double()
        a = g * torch.sigmoid(g) if case["act"] == "silu" else torch.nn.functional.gelu(g, approximate="tanh")
        y = y.index_add(0, t, w[t, k, None] * ((a * (x[t] @ s["up"][j].double())) @ s["down"][j].double()))
    return {"y": y, "experts": experts, "weights": w}
