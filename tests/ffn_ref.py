"""Plain float64 references of the operators in include/a2av_ffn.h, on the CPU, and the error bounds the GPU tests
use.  Nothing here is shared with the library.

Bounds.  u is the output type's unit roundoff (2^-8 bf16, 2^-11 fp16; half of the gap to the next value is at most
u times the value) and step its smallest subnormal.  A tensor-core product of length K with fp32 accumulation is
taken to be within (K + 8) 2^-23 sum |a b| of the exact one (one rounding or truncation a term).  fp32 chains of a
row (sum of squares, reciprocal root, exponential, quotient) are within 2^-18 relative: a block sum adds at most 64
values a thread and ten levels, and the special functions are good to a few units of 2^-24 (the exponential to about
|z| 2^-23, |z| < 32 where its term counts).
"""

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
STEP = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -24}
CHAIN = 2.0 ** -18
F8 = {"e4m3fn": (torch.float8_e4m3fn, 8, 448.0, 3, -6), "e5m2": (torch.float8_e5m2, 15, 57344.0, 2, -14)}
QMAX = {"e4m3fn": 448.0, "e5m2": 57344.0, "int8": 127.0}


# ------------------------------------------------------------------ norm


def rms_norm(x, residual, gamma, eps):
    s = x.double() + (residual.double() if residual is not None else 0.0)
    rstd = 1.0 / torch.sqrt((s * s).mean(1) + eps)
    return s, s * rstd[:, None] * gamma.double(), rstd


def rms_norm_backward(dy, dh, h, gamma, rstd):
    dy, h, gamma, rstd = dy.double(), h.double(), gamma.double(), rstd.double()
    a, n = dy * gamma, h * rstd[:, None]
    dx = rstd[:, None] * (a - n * (a * n).mean(1, keepdim=True))
    if dh is not None:
        dx = dx + dh.double()
    return dx, (dy * n).sum(0)


# ------------------------------------------------------------------ gated block


def _z(g, name):
    """Both activations are g * sigmoid(z); (1 + tanh(t)) / 2 = sigmoid(2t), without the cancellation of 1 + tanh(t)."""
    return g if name == "silu" else 2.0 * 0.7978845608028654 * (g + 0.044715 * g ** 3)


def act(g, name):
    return g / (1.0 + torch.exp(-_z(g, name)))


def act_slope(g, name):
    z = _z(g, name)
    s, rest = 1.0 / (1.0 + torch.exp(-z)), 1.0 / (1.0 + torch.exp(z))
    dz = 1.0 if name == "silu" else 2.0 * 0.7978845608028654 * (1.0 + 3 * 0.044715 * g * g)
    return s + g * dz * s * rest


def arrival_index(counts, W, e):
    """Arrival row of each expert-major row, and the experts' row counts."""
    starts, at = [], 0
    for c in counts:
        starts.append(at)
        at += int(c)
    order, sizes = [], []
    for j in range(e):
        n = 0
        for w in range(W):
            c = int(counts[w * e + j])
            order.extend(range(starts[w * e + j], starts[w * e + j] + c))
            n += c
        sizes.append(n)
    return torch.tensor(order, dtype=torch.int64), sizes


def per_expert(fn, sizes, *mats):
    """fn(expert, that expert's rows of each matrix), stacked."""
    out, at = [], 0
    for j, n in enumerate(sizes):
        out.append(fn(j, *[m[at:at + n] for m in mats]))
        at += n
    return out


def gated(x, counts, W, e, wg, wu, name):
    """Expert-major G, U, h and the bound on h's error before its rounding."""
    idx, sizes = arrival_index(counts, W, e)
    xe, wg, wu = x.double()[idx], wg.double(), wu.double()
    cat = lambda parts: torch.cat(parts) if parts else xe.new_zeros(0, wg.shape[2])
    G = cat(per_expert(lambda j, r: r @ wg[j], sizes, xe))
    U_ = cat(per_expert(lambda j, r: r @ wu[j], sizes, xe))
    slack = (xe.shape[1] + 8) * 2.0 ** -23
    eg = slack * cat(per_expert(lambda j, r: r.abs() @ wg[j].abs(), sizes, xe))
    eu = slack * cat(per_expert(lambda j, r: r.abs() @ wu[j].abs(), sizes, xe))
    a = act(G, name)
    h = a * U_
    # slopes of both activations stay below 1.13
    return {"xe": xe, "sizes": sizes, "idx": idx, "G": G, "U": U_, "eg": eg, "eu": eu, "h": h,
            "eh": 1.13 * eg * (U_.abs() + eu) + a.abs() * eu + CHAIN * h.abs()}


def gated_backward(f, dh, wg, wu, name, dtype):
    """dX (rank-major), dWg, dWu and the bounds on their errors before rounding.  dG and dU are rounded to the element
    type on the way (u each), and come from G and U that are eg and eu off (second derivatives below 1)."""
    dh, wg, wu = dh.double(), wg.double(), wu.double()
    s, a = act_slope(f["G"], name), act(f["G"], name)
    dG, dU = dh * f["U"] * s, dh * a
    u, st = U[dtype], STEP[dtype]
    eG = u * dG.abs() + st + (1 + u) * (dh.abs() * (1.13 * f["eu"] + (f["U"].abs() + f["eu"]) * f["eg"]) + CHAIN * (
        dh * f["U"]).abs())
    eU = u * dU.abs() + st + (1 + u) * (dh.abs() * 1.13 * f["eg"] + CHAIN * dU.abs())
    return _two_sided(f["xe"], f["sizes"], f["idx"], [(dG, eG, wg), (dU, eU, wu)])


def gmm_backward(xe, counts, W, e, dy, w):
    idx, sizes = arrival_index(counts, W, e)
    dy = dy.double()
    (dx, ex), grads = _two_sided(xe.double(), sizes, idx, [(dy, torch.zeros_like(dy), w.double())])
    return (dx, ex), grads


def _two_sided(xe, sizes, idx, terms):
    e, H1, N = terms[0][2].shape
    dxe, exe = xe.new_zeros(xe.shape), xe.new_zeros(xe.shape)
    grads = []
    for D, E, w in terms:
        dW, eW = [], []
        at = 0
        for j, n in enumerate(sizes):
            r = slice(at, at + n)
            dxe[r] += D[r] @ w[j].t()
            exe[r] += E[r] @ w[j].abs().t() + (len(terms) * N + 8) * 2.0 ** -23 * ((D[r].abs() + E[r]) @ w[j].abs().t())
            dW.append(xe[r].t() @ D[r])
            eW.append(xe[r].abs().t() @ E[r] + (n + 8) * 2.0 ** -23 * (xe[r].abs().t() @ (D[r].abs() + E[r])))
            at += n
        grads.append((torch.stack(dW), torch.stack(eW)))
    dx, ex = torch.zeros_like(dxe), torch.zeros_like(exe)
    dx[idx], ex[idx] = dxe, exe
    return (dx, ex), grads


# ------------------------------------------------------------------ comparisons


def assert_rounded(got, ref, err, what):
    """got, of a 16-bit type, is the rounding of a value within err of ref."""
    u, step = U[got.dtype], STEP[got.dtype]
    g = got.double().cpu()
    assert g.shape == ref.shape, (what, g.shape, ref.shape)
    nan = torch.isnan(ref)
    assert torch.equal(torch.isnan(g), nan), what
    lim = err * (1 + u) + u * ref.abs() + step
    bad = ~nan & ~((g - ref).abs() <= lim) & ~(g == ref)
    assert not bad.any(), (what, int(bad.sum()), torch.nonzero(bad)[:4].tolist(), g[bad][:4].tolist(),
                           ref[bad][:4].tolist(), lim[bad][:4].tolist())


def decode(codes, qtype):
    c = codes.cpu()
    return c.view(torch.int8).double() if qtype == "int8" else c.view(F8[qtype][0]).double()


def assert_codes(codes, scales, ref, rel, qtype, mode, what):
    """codes and scales stand for a value within rel of ref (relative, fp32 chain) rounded to the format."""
    rows, n = ref.shape
    block = 32 if mode == "mx" else 128
    b = ref.reshape(rows, n // block, block)
    c = decode(codes, qtype).reshape(b.shape)
    amax = b.abs().amax(2)
    finite = torch.isfinite(b).all(2)
    if mode == "mx":
        emax = F8[qtype][1]
        sc = scales.cpu().to(torch.int64).reshape(amax.shape)
        assert torch.equal(sc == 255, ~finite), what
        want = lambda m: (torch.floor(torch.log2(m.clamp_min(2.0 ** -140))) - emax).clamp(-127, 127).to(torch.int64) + 127
        lo, hi = want(amax * (1 - rel)), want(amax * (1 + rel))
        assert bool(((sc >= lo) & (sc <= hi))[finite].all()), what
        scale = torch.exp2(sc.double() - 127)
        top = F8[qtype][2]
    else:
        top = QMAX[qtype]
        scale = scales.cpu().double().reshape(amax.shape)
        assert torch.equal(torch.isnan(scale), ~finite), what
        m = amax.clamp_min(2.0 ** -100) / top
        assert bool(((scale - m).abs() <= m * (rel + 2.0 ** -22))[finite].all()), what
    if qtype == "int8":
        assert bool((c[~finite] == 0).all()), what
    else:
        assert bool(torch.isnan(c[~finite]).all()), what
    v = (b / scale[..., None])
    sat = v.clamp(-top, top)
    slack = v.abs() * (rel + 2.0 ** -21)
    if qtype == "int8":
        half = torch.full_like(v, 0.5)
    else:  # half of the gap to the next code at the value or just above it
        _, _, _, mant, emin = F8[qtype]
        ex = torch.floor(torch.log2((v.abs() + slack).clamp_min(2.0 ** emin))).clamp_min(emin)
        half = torch.exp2(ex - mant - 1)
    bad = ~((c - sat).abs() <= half + slack) & finite[..., None]
    assert not bad.any(), (what, int(bad.sum()), torch.nonzero(bad)[:4].tolist(), c[bad][:4], v[bad][:4])
