"""Plain 64-bit forms of the experts' operators with the error each allows, for the GPU tests.

Every form returns (value, allowance): the value in float64 from the operator's
definition, and a bound on what a binary32 evaluation of it may be off before
the last rounding, from these facts: a sum of n binary32 products is off by at
most (n + 8) * 2^-23 of the sum of their magnitudes whatever the order
(products of bf16 values and 8- or 4-bit codes are exact; twice the unit
roundoff covers accumulators that truncate); sigma(z) = 1 / (1 + exp(-z)) by
exp2 of a rounded product is off by (|z| + 8) * 2^-23 relative. A rounding to
the output type adds half a step, finfo(type).eps / 2 of the value.
"""
import torch

U = 2.0 ** -23
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def codes_e2m1(w):
    """The values of packed e2m1 bytes, the low half first."""
    code = torch.stack([w & 15, w >> 4], -1).flatten(-2).long()
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device=w.device)
    return table[code]


def values(w, scales, kind):
    """Rows or weights as float64 values ("bf16", "fp32", "fp8" or "fp4" with scales or None)."""
    if kind == "fp4":
        v = codes_e2m1(w)
    elif kind == "fp8":
        v = w.view(torch.float8_e4m3fn).double()
    else:
        v = w.double()
    return v if scales is None else v * scales.double().repeat_interleave(128, -1)


def product(x, dx, w):
    """x w^T with the error of x carried along: rows x [n, K] off by dx, a matrix [N, K]."""
    y = x @ w.T
    size = x.abs() @ w.abs().T
    return y, dx @ w.abs().T + (x.shape[1] + 8) * U * (size + dx @ w.abs().T)


def sigmoid(z):
    return torch.sigmoid(z), torch.sigmoid(z) * (z.abs() + 8) * U


def gated(g, dg, u, du):
    """silu(g) * u; the slope of silu is at most 1.1. The relative bounds hold for normal
    numbers; below 2^-126 a binary32 rounding is off by half of the smallest step, 2^-150,
    whatever the value: so silu(g) by 2^-149 (a division and a product), which u then scales."""
    s, ds = sigmoid(g)
    h = g * s * u
    dh = (1.1 * dg + g.abs() * ds) * (u.abs() + du) + (g * s).abs() * du + 4 * U * h.abs() + 2.0 ** -149 * (u.abs() + 1)
    return h, dh


def gated_backward(dh, g, u):
    s, ds = sigmoid(g)
    a = 1 + g * (1 - s)
    da = g.abs() * (ds + U) + 2 * U * (1 + g.abs())
    d = torch.cat([dh * u * s * a, dh * g * s], -1)
    e = torch.cat([(dh * u).abs() * (s * da + ds * a.abs() + 4 * U * s * a.abs()),
                   (dh * g).abs() * (ds + 4 * U * s)], -1)
    return d, e


def checkpoint(v):
    """(codes as float64 values, scales) of rows by the definition, 128 values a group."""
    g = v.double().unflatten(-1, (-1, 128))
    size = g.abs()
    top = torch.where(torch.isfinite(size), size, 0.0).amax(-1)
    p = torch.full_like(top, -126.0)
    # the smallest p >= -126 with top <= 448 * 2^p, by the exponent and an exact comparison
    m, e = torch.frexp(top)
    q = (e - 9).double()
    q = torch.where(top > 448 * torch.exp2(q), q + 1, q)
    p = torch.where(top > 0, q.clamp(min=-126), p)
    scale = torch.exp2(p)
    scaled = torch.where(torch.isfinite(g), g / scale[..., None], float("nan"))
    # e4m3, round to nearest even: steps of 2^-3 of the binade, 2^-9 below 2^-6
    m, e = torch.frexp(scaled.abs().clamp(min=2.0 ** -6))
    step = torch.exp2((e - 4).double())
    code = torch.round(scaled / step) * step
    return code.flatten(-2), scale


def layer(x, idx, probs, bias, w_in, in_scales, w_out, out_scales, kind, E, I):
    """The expert layer, entry by entry in groups of an expert."""
    T, K = idx.shape
    H = x.shape[1]
    out = torch.zeros(T, H, dtype=torch.float64, device=x.device)
    err, size = torch.zeros_like(out), torch.zeros_like(out)
    for e in torch.unique(idx).tolist():
        if e < 0 or e >= E:
            continue
        t, k = torch.nonzero(idx == e, as_tuple=True)
        xe = x[t].double()
        z, dz = product(xe, torch.zeros_like(xe), values(w_in[e], None if in_scales is None else in_scales[e], kind))
        h, dh = gated(z[:, :I], dz[:, :I], z[:, I:], dz[:, I:])
        dh = dh + 2.0 ** -16 * h.abs()  # h as a high and a low bf16 part: 2^-8 of 2^-8, and the cut of the low
        y, dy = product(h, dh, values(w_out[e], None if out_scales is None else out_scales[e], kind))
        p = (torch.ones(len(t), 1, dtype=torch.float64, device=x.device) if probs is None
             else probs[t, k].double()[:, None])
        out.index_add_(0, t, y * p)
        err.index_add_(0, t, dy * p.abs())
        size.index_add_(0, t, (y * p).abs())
    if bias is not None:
        out, size = out + bias.double(), size + bias.double().abs()
    return out, err + (K + 2) * U * size


def near(got, want, allowed, dtype):
    """Every element within its allowance and half a step of the output type."""
    half = torch.finfo(dtype).eps / 2
    tiny = torch.finfo(dtype).tiny
    off = (got.double() - want).abs()
    bound = allowed * (1 + half) + half * want.abs() + tiny * torch.finfo(dtype).eps
    bad = ~(off <= bound)
    assert not bool(bad.any()), (f"{int(bad.sum())} of {off.numel()} off: worst {float((off - bound).max()):.3g} "
                                 f"over, at {torch.nonzero(bad)[0].tolist()}")
