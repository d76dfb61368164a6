"""Plain 64-bit forms of the router's operators with the error each allows, for the GPU tests.

Bounds on a binary32 evaluation before the last rounding, with U = 2^-23 (twice the unit roundoff): an
exponential of a difference z by exp2 of a rounded product is off by (|z| + 8) U relative, a sigmoid the
same; a row's sum of up to 1024 positive terms, added 16 deep in a lane and 6 deep across lanes, by 22 U
more. So a score or probability is off by at most (spread + 40) U relative, where spread is the largest
|l - max l| (softmax) or |l| (sigmoid) of the row's finite logits, twice where a quotient has the error
above and below it. What is added up with both signs is off by that much of the sum of magnitudes. A sum
of up to 256 tokens adds 264 U.
"""
import torch

U = 2.0 ** -23
INF = float("inf")


def scores(l, scoring):
    """(scores, probabilities, log of the sum of exponentials, spread) of logits in 64 bits."""
    finite = torch.isfinite(l)
    safe = torch.where(finite, l, 0.0)
    none = (l == -INF).all(1, keepdim=True)
    base = torch.where(none, torch.zeros_like(l), l)
    soft = torch.where(none, 0.0, torch.softmax(base, 1))
    lse = torch.where(none[:, 0], 0.0, torch.logsumexp(base, 1))
    if scoring == "softmax":
        top = torch.where(finite, l, -INF).amax(1, keepdim=True)
        spread = torch.where(finite, torch.where(torch.isfinite(top), top, 0.0) - safe, 0.0).amax(1)
        return soft, soft, lse, spread.clamp(max=110.0)
    s = torch.sigmoid(l)
    # quotients of sigmoids that underflow: log s = -log(1 + exp(-l))
    p = torch.where(none, 0.0, torch.softmax(torch.where(none, torch.zeros_like(l), torch.nn.functional.logsigmoid(l)), 1))
    return s, p, lse, safe.abs().amax(1).clamp(max=220.0)


def choose(l, K, scoring, bias=None, mask=None):
    if bias is None:
        key = l.clone()
    else:
        key = scores(l, scoring)[0] + bias.double()
        key = torch.where(l == -INF, -INF, key)
    key = torch.where(torch.isnan(key) | torch.isnan(l), -INF, key)
    if mask is not None:
        key = torch.where(mask[:, None] != 0, key, -INF)
    v, ids = torch.sort(key, dim=1, descending=True, stable=True)
    return torch.where(v[:, :K] == -INF, -1, ids[:, :K])


def quotients(l, ids, scoring):
    """Of each entry its score over the sum of its token's entries' (0 where that sum is 0)."""
    real = ids >= 0
    v = l.gather(1, ids.clamp(min=0))
    log = v if scoring == "softmax" else torch.nn.functional.logsigmoid(v)
    log = torch.where(real, log, -INF)
    dead = (log == -INF).all(1, keepdim=True)
    return torch.where(dead, 0.0, torch.softmax(torch.where(dead, torch.zeros_like(log), log), 1))


def weights(l, ids, scoring, normalize, scale):
    real = ids >= 0
    s, _, _, spread = scores(l, scoring)
    w = quotients(l, ids, scoring) if normalize else torch.where(real, s.gather(1, ids.clamp(min=0)), 0.0)
    # An exponential below 2^-126 may be 0 (the instruction gives no subnormal numbers). It is divided by a sum that
    # holds a term of at least 1/2 (exp(0), or a sigmoid of its reference): off by at most 2^-125, times the scale.
    return w * scale, w * abs(scale) * ((2 * spread + 90) * U)[:, None] + 2.0 ** -125 * abs(scale)


def sequences(T, seq_offsets, device):
    t = torch.arange(T, device=device)
    if seq_offsets is None:
        return torch.zeros_like(t), torch.ones_like(t, dtype=torch.bool), 1
    o = seq_offsets.long().to(device)
    s = torch.searchsorted(o, t, right=True) - 1
    S = o.numel() - 1
    return s.clamp(0, S - 1), (s >= 0) & (s < S), S


def statistics(l, ids, scoring, seq_offsets):
    """(counts, seq_tokens, (balance, allowance), (z, allowance))."""
    T, E = l.shape
    K = ids.shape[1]
    _, p, lse, spread = scores(l, scoring)
    seq, on, S = sequences(T, seq_offsets, l.device)
    real = ids >= 0
    on = on & real.any(1)
    at = (seq[:, None] * E + ids)[real & on[:, None]]
    counts = torch.bincount(at, minlength=S * E).view(S, E)
    n = torch.bincount(seq[on], minlength=S)
    full, total = int((n > 0).sum()), int(n.sum())
    tokens = torch.cat([n, torch.tensor([full, total], device=n.device)])
    P = torch.zeros(S, E, dtype=torch.float64, device=l.device).index_add_(0, seq[on], p[on])
    m = n.double().clamp(min=1)[:, None]
    balance = float((E * counts / (K * m) * P / m).sum() / max(full, 1))
    err = float(spread[on].max()) if total else 0.0
    z = float((lse[on] ** 2).sum() / max(total, 1))
    dz = float(((2 * lse.abs() * (lse.abs() + spread + 60) + lse ** 2 * 264)[on]).sum() / max(total, 1)) * U
    return counts, tokens, (balance, balance * (2 * err + 90 + 264) * U), (z, dz)


def backward(l, ids, scoring, normalize, scale, dw, seq_offsets, counts, tokens, db, dz):
    """(d_logits, allowance): the formulas, with the sum of the magnitudes that are added."""
    T, E = l.shape
    K = ids.shape[1]
    s, p, lse, spread = scores(l, scoring)
    real = ids >= 0
    at = ids.clamp(min=0)
    d = torch.zeros_like(l)
    size = torch.zeros_like(l)
    if dw is not None:
        dw = torch.where(real, dw.double() * scale, 0.0)
        if normalize:
            q = quotients(l, ids, scoring)
            e = q * (dw - (q * dw).sum(1, keepdim=True))
            m = q * (dw.abs() + (q * dw.abs()).sum(1, keepdim=True))
            if scoring == "sigmoid":
                far = torch.sigmoid(-l).gather(1, at)
                e, m = e * far, m * far
            d.scatter_add_(1, at, torch.where(real, e, 0.0))
            size.scatter_add_(1, at, torch.where(real, m, 0.0))
        elif scoring == "sigmoid":
            e = dw * (s * torch.sigmoid(-l)).gather(1, at)
            d.scatter_add_(1, at, torch.where(real, e, 0.0))
            size.scatter_add_(1, at, torch.where(real, e.abs(), 0.0))
        else:
            dp = torch.zeros_like(l).scatter_add_(1, at, dw)
            mp = torch.zeros_like(l).scatter_add_(1, at, dw.abs())
            d = p * (dp - (p * dp).sum(1, keepdim=True))
            size = p * (mp + (p * mp).sum(1, keepdim=True))
    seq, on, _ = sequences(T, seq_offsets, l.device)
    on = (on & real.any(1))[:, None]
    if db is not None:
        n = tokens[:-2].double().clamp(min=1)[:, None]
        g = (db * counts.double() * E / (K * n * n * max(int(tokens[-2]), 1)))[seq]
        far = torch.sigmoid(-l) if scoring == "sigmoid" else torch.ones_like(l)
        d = d + torch.where(on, p * far * (g - (p * g).sum(1, keepdim=True)), 0.0)
        size = size + torch.where(on, p * far * (g.abs() + (p * g.abs()).sum(1, keepdim=True)), 0.0)
    if dz is not None:
        v = 2 * dz / max(int(tokens[-1]), 1) * p
        d = d + torch.where(on, v * lse[:, None], 0.0)
        size = size + torch.where(on, v.abs() * (lse.abs() + 1)[:, None], 0.0)
    return d, size * ((4 * spread + 160) * U)[:, None] + 2.0 ** -120


def near(got, want, allowed, dtype):
    """Every element within its allowance and half a step of the output type."""
    half = torch.finfo(dtype).eps / 2
    off = (got.double() - want).abs()
    bound = allowed * (1 + half) + half * want.abs() + torch.finfo(dtype).tiny * torch.finfo(dtype).eps
    bad = ~(off <= bound)
    assert not bool(bad.any()), (f"{int(bad.sum())} of {off.numel()} off: worst {float((off - bound).max()):.3g} "
                                 f"over, at {torch.nonzero(bad)[0].tolist()}")
