"""Cases of the router's and the 8-bit integer operators: what a call of each takes, its plain form and its definition in 64 bits.

ep_router            scores of a router's logits, the chosen experts, their weights, per-expert counts, balance and z loss
ep_router_backward   the logits' gradient from the weights' and the losses'
ep_quantize_rows     rows to 8-bit integers with one scale per row
ep_swiglu_quantize   the experts' activation, quantised the same way
ep_quantized_matmul  per-expert products of 8-bit integers with a scale per row and per channel

Rows of expert e are [offsets[e], offsets[e] + counts[e]) of an expand buffer. Tokens of sequence s are
[seq_offsets[s], seq_offsets[s + 1]); a token takes part in the statistics if one of its ids is in [0, E).
"""
import math

import torch

own = False

LEAST = 2.0 ** -100  # a row's largest magnitude counts as at least this


def listed():
    route, back = {"op": "router"}, {"op": "router_backward"}
    quant, gated, mm = {"op": "quantize_rows"}, {"op": "swiglu_quantize"}, {"op": "quantized_matmul"}
    return [
        # a decode step of 128 tokens, selection by score + bias: latency counts, no statistics
        {"name": "router_decode", **route, "T": 128, "E": 256, "K": 8, "S": 0, "rows": "fp32", "scoring": "sigmoid",
         "bias": True, "normalize": True, "given": False, "masked": 0.0, "excluded": 0.0},
        # a training batch of 4096 tokens, balance loss over the whole batch and z loss
        {"name": "router_train", **route, "T": 4096, "E": 256, "K": 8, "S": 1, "rows": "fp32", "scoring": "softmax",
         "bias": False, "normalize": True, "given": False, "masked": 0.0, "excluded": 0.0},
        # packed sequences with padding, a loss per sequence, selection by score + bias
        {"name": "router_train_packed", **route, "T": 32768, "E": 256, "K": 8, "S": 37, "rows": "fp32",
         "scoring": "sigmoid", "bias": True, "normalize": True, "given": False, "masked": 0.03, "excluded": 0.0},
        # backward of a small odd batch whose ids the caller chose, bf16 logits
        {"name": "router_back_odd", **back, "T": 1021, "E": 60, "K": 4, "S": 1, "rows": "bf16", "scoring": "softmax",
         "bias": False, "normalize": False, "given": True, "masked": 0.1, "excluded": 0.0},
        # backward of the packed batch
        {"name": "router_back_packed", **back, "T": 32768, "E": 256, "K": 8, "S": 37, "rows": "fp32",
         "scoring": "sigmoid", "bias": True, "normalize": True, "given": False, "masked": 0.03, "excluded": 0.0},
        # the tokens of a decode step, a scale row per token as dispatch moves it
        {"name": "quantize_decode", **quant, "T": 128, "K": 1, "E": 1, "A": 1, "width": 7168, "rows": "bf16",
         "copies": 56, "routing": "uniform"},
        # the prefill batch's expand buffer: 32768 rows among alignment padding
        {"name": "quantize_expand", **quant, "T": 4096, "K": 8, "E": 256, "A": 128, "width": 7168, "rows": "bf16",
         "copies": 1, "routing": "uniform"},
        # activation of a small odd fp32 batch
        {"name": "swiglu_quantize_small", **gated, "T": 61, "K": 6, "E": 64, "A": 1, "width": 1408, "rows": "fp32",
         "copies": 1, "routing": "zipf"},
        # activation of the prefill batch
        {"name": "swiglu_quantize_prefill", **gated, "T": 4096, "K": 8, "E": 256, "A": 128, "width": 2048,
         "rows": "bf16", "copies": 1, "routing": "uniform"},
        # one dense projection of one token (a shared expert)
        {"name": "matmul_one_row", **mm, "T": 1, "K": 1, "E": 1, "A": 1, "in": 7168, "out": 4096, "y": "bf16",
         "routing": "uniform"},
        # the up projection of a decode batch: every expert's weights for a few rows each
        {"name": "matmul_decode", **mm, "T": 128, "K": 8, "E": 64, "A": 1, "in": 7168, "out": 4096, "y": "bf16",
         "routing": "zipf"},
        # the up projection of a prefill batch, about 512 rows an expert
        {"name": "matmul_prefill", **mm, "T": 4096, "K": 8, "E": 64, "A": 128, "in": 7168, "out": 4096, "y": "bf16",
         "routing": "uniform"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["router", "router_backward", "quantize_rows", "swiglu_quantize", "quantized_matmul"])
    E = _log_int(rng, 1, 256)
    if op in ("router", "router_backward"):
        E = _log_int(rng, 2, 1024)
        T = _log_int(rng, 1, 32768 * 256 // max(E, 256))
        scoring = rng.choice(["softmax", "sigmoid"])
        given = rng.random() < 0.3
        return {"op": op, "T": T, "E": E, "K": min(E, rng.choice([1, 2, 4, 6, 8])),
                "S": _log_int(rng, 1, max(1, T // 4)) if op == "router_backward" else rng.choice([0, 1, _log_int(rng, 1, max(1, T // 4))]),
                "rows": rng.choice(["bf16", "fp32"]), "scoring": scoring, "bias": not given and rng.random() < 0.4,
                "normalize": rng.random() < 0.6, "given": given, "masked": rng.choice([0.0, 0.1]),
                "excluded": rng.choice([0.0, 0.2])}
    K = min(E, rng.choice([1, 2, 4, 6, 8]))
    case = {"op": op, "K": K, "E": E, "A": rng.choice([1, 16, 128]), "routing": rng.choice(["uniform", "zipf"])}
    if op == "quantized_matmul":
        return {**case, "E": min(E, 64), "K": min(K, E, 64), "T": _log_int(rng, 1, 4096), "in": _log_int(rng, 2, 448) * 16,
                "out": _log_int(rng, 8, 512) * 8, "y": rng.choice(["bf16", "fp32"])}
    return {**case, "T": _log_int(rng, 1, 2048), "width": _log_int(rng, 4, 448 if op == "quantize_rows" else 128) * 16,
            "rows": rng.choice(["bf16", "fp32"]), "copies": rng.choice([1, 1, 7])}


# ---------------------------------------------------------------------------------------- inputs

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _normal(shape, gen, std=1.0, kind="fp32"):
    return torch.empty(shape, dtype=TYPES[kind], device="cuda").normal_(0.0, std, generator=gen)


def _expand(case, gen):
    """The routing arrays of an expand buffer: counts, offsets, rows of the buffer, and the most rows of an expert."""
    T, K, E, A = (case[k] for k in ("T", "K", "E", "A"))
    noise = torch.rand(T, E, generator=gen, device="cuda", dtype=torch.float64).clamp_(1e-12, 1 - 1e-12)
    if case["routing"] == "zipf":  # the K largest of log-popularity + Gumbel noise
        order = torch.randperm(E, generator=gen, device="cuda").double()
        noise = (-1.1 * torch.log1p(order))[None, :] - torch.log(-torch.log(noise))
    counts = torch.bincount(noise.argsort(dim=1, descending=True)[:, :K].reshape(-1), minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum((counts + A - 1) // A * A, 0)
    return counts.to(torch.int32), offsets.to(torch.int32), T * K + E * (A - 1), int(counts.max())


def _router_state(case, gen, s):
    T, E, K, S = (case[k] for k in ("T", "E", "K", "S"))
    popular = _normal((1, E), gen, 0.5)  # some experts are liked more than others
    logits = _normal((T, E), gen, 1.5) + popular
    if case["excluded"]:
        out = torch.rand(E, generator=gen, device="cuda") < case["excluded"]
        out[0] = False  # one stays
        logits[:, out] = -math.inf
    s["logits"] = logits.to(TYPES[case["rows"]])
    s["bias"] = _normal((E,), gen, 0.05) - 0.1 * popular[0] if case["bias"] else None
    kept = torch.rand(T, generator=gen, device="cuda") >= case["masked"]
    s["mask"] = kept.to(torch.uint8) if case["masked"] and not case["given"] else None
    cut = torch.sort(torch.randint(0, T + 1, (max(S - 1, 0),), generator=gen, device="cuda")).values
    ends = torch.tensor([0, T], device="cuda")
    s["seq_offsets"] = torch.cat([ends[:1], cut, ends[1:]]).to(torch.int32) if S > 1 else None
    s["scale"] = 2.5
    s["idx"] = torch.randint(0, E, (T, K), generator=gen, device="cuda", dtype=torch.int32)
    s["idx"][~kept] = -1  # given: ids of tokens that are left out
    s["weights"] = torch.empty(T, K, device="cuda")
    s["counts"] = torch.empty(max(S, 1), E, dtype=torch.int32, device="cuda")
    s["seq_tokens"] = torch.empty(max(S, 1) + 2, dtype=torch.int32, device="cuda")
    s["losses"] = torch.empty(2, device="cuda")
    s["workspace"] = torch.empty((T // 16 + S + 64) * (E + 16) * 8, dtype=torch.uint8, device="cuda")
    if case["op"] == "router_backward":
        # what the forward pass left: ids, counts and numbers of tokens
        ids = s["idx"].long() if case["given"] else _choose(s, case)
        s["idx"] = ids.to(torch.int32)
        seq, inside = _sequences(s, case)
        real, inside = ids >= 0, inside & (ids >= 0).any(1)
        at = (seq[:, None] * E + ids)[real & inside[:, None]]
        s["counts"] = torch.bincount(at, minlength=max(S, 1) * E).view(-1, E).to(torch.int32)
        tokens = torch.bincount(seq[inside], minlength=max(S, 1))
        s["seq_tokens"] = torch.cat([tokens, (tokens > 0).sum()[None], tokens.sum()[None]]).to(torch.int32)
        s["d_weights"] = _normal((T, K), gen, 1.0 / T)
        s["d_losses"] = torch.tensor([1e-2, 1e-3], device="cuda")
        s["d_logits"] = torch.empty_like(s["logits"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op in ("router", "router_backward"):
        _router_state(case, gen, s)
        return s
    s["counts"], s["offsets"], s["cap"], s["most"] = _expand(case, gen)
    cap = s["cap"]
    if op == "quantized_matmul":
        E, C, N = case["E"], case["in"], case["out"]
        # codes as quantising normal rows leaves them: their largest magnitude is about 4 standard deviations
        s["x"] = _normal((cap, C), gen, 32.0).round_().clamp_(-127, 127).to(torch.int8)
        s["w"] = torch.empty(E, N, C, dtype=torch.int8, device="cuda")
        for e in range(E):
            s["w"][e] = _normal((N, C), gen, 32.0).round_().clamp_(-127, 127).to(torch.int8)
        s["x_scales"] = torch.empty(cap, 1, device="cuda").uniform_(0.02, 0.05, generator=gen)
        s["w_scales"] = torch.empty(E, N, device="cuda").uniform_(0.02, 0.05, generator=gen) * C ** -0.5
        s["y"] = torch.zeros(cap, N, dtype=TYPES[case["y"]], device="cuda")
        return s
    W = case["width"]
    s["x"] = _normal((cap, W if op == "quantize_rows" else 2 * W), gen, 1.5, case["rows"])
    s["codes"] = torch.zeros(cap, W, dtype=torch.int8, device="cuda")
    s["scales"] = torch.zeros(cap, case["copies"], device="cuda")
    return s


# ---------------------------------------------------------------------------------------- plain forms

def _sequences(s, case):
    """For each token its sequence, and whether it has one."""
    T = case["T"]
    t = torch.arange(T, device=s["logits"].device)
    if s["seq_offsets"] is None:
        return torch.zeros_like(t), torch.ones_like(t, dtype=torch.bool)
    begin = s["seq_offsets"].long()
    seq = torch.searchsorted(begin, t, right=True) - 1
    return seq.clamp(0, begin.numel() - 2), (t >= begin[0]) & (t < begin[-1])


def _choose(s, case):
    """The K experts of each token by descending logit, or score + bias (in 64 bits), ties by ascending id; -1: none left."""
    key = s["logits"].double()
    if s["bias"] is not None:
        score = torch.softmax(key, 1) if case["scoring"] == "softmax" else 1 / (1 + torch.exp(-key))
        key = torch.where(key == -math.inf, key, score + s["bias"].double())
    if s["mask"] is not None:
        key = torch.where(s["mask"][:, None] != 0, key, -math.inf)
    v, ids = torch.sort(key, dim=1, descending=True, stable=True)
    return torch.where(v[:, :case["K"]] == -math.inf, -1, ids[:, :case["K"]])


def _scores(s, case):
    """(scores, probabilities, log of the sum of exponentials) in 32 bits."""
    l = s["logits"].float()
    if case["scoring"] == "sigmoid":
        v = 1 / (1 + torch.exp(-l))
        return v, v / v.sum(1, keepdim=True), None
    m = l.amax(1, keepdim=True)
    ex = torch.exp(l - m)
    total = ex.sum(1, keepdim=True)
    return ex / total, ex / total, torch.log(total) + m


def _plain_router(s, case):
    T, E, K, S = (case[k] for k in ("T", "E", "K", "S"))
    ids = s["idx"].long() if case["given"] else _choose(s, case)
    real = ids >= 0
    score, p, lse = _scores(s, case)
    w = torch.where(real, score.gather(1, ids.clamp(min=0)), 0.0)
    if case["normalize"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, 1.0)
    out = {"idx": ids.to(torch.int32), "weights": w * s["scale"]}
    if S == 0:
        return out
    seq, inside = _sequences(s, case)
    inside = inside & real.any(1)
    at = (seq[:, None] * E + ids)[real & inside[:, None]]
    counts = torch.bincount(at, minlength=S * E).view(S, E)
    tokens = torch.bincount(seq[inside], minlength=S)
    n = tokens.double().clamp(min=1)[:, None]
    upto = torch.cat([torch.zeros(1, E, dtype=torch.float64, device=w.device),
                      torch.where(inside[:, None], p, 0.0).cumsum(0, dtype=torch.float64)])
    begin = torch.tensor([0, T], device=w.device) if s["seq_offsets"] is None else s["seq_offsets"].long()
    total = upto[begin[1:]] - upto[begin[:-1]]
    full = (tokens > 0).sum()
    losses = [(E * counts / (K * n) * total / n).sum() / full.clamp(min=1)]
    if lse is not None:
        losses.append((lse[inside].double() ** 2).sum() / tokens.sum().clamp(min=1))
    return {**out, "counts": counts.to(torch.int32), "seq_tokens": torch.cat([tokens, full[None], tokens.sum()[None]]).to(torch.int32),
            "losses": torch.stack(losses).float()}


def _plain_backward(s, case):
    E, K = case["E"], case["K"]
    ids = s["idx"].long()
    real = ids >= 0
    score, p, lse = _scores(s, case)
    softmax = case["scoring"] == "softmax"
    dw = torch.where(real, s["d_weights"] * s["scale"], 0.0)
    chosen = torch.where(real, score.gather(1, ids.clamp(min=0)), 0.0)
    if case["normalize"]:
        total = chosen.sum(1, keepdim=True)
        q = chosen / torch.where(total > 0, total, 1.0)
        d = q * (dw - (q * dw).sum(1, keepdim=True))
        if not softmax:
            d = d * (1 - chosen)
    else:
        d = dw * chosen if softmax else dw * chosen * (1 - chosen)
    out = torch.zeros_like(score).scatter_add_(1, ids.clamp(min=0), d)
    if softmax and not case["normalize"]:
        out = out - p * d.sum(1, keepdim=True)
    seq, inside = _sequences(s, case)
    inside = (inside & real.any(1))[:, None]
    n = s["seq_tokens"][:-2].double().clamp(min=1)[:, None]
    g = (s["counts"].double() * E / (K * n * n * s["seq_tokens"][-2].clamp(min=1))).float() * s["d_losses"][0]
    g = g[seq]
    if softmax:
        z = 2 * lse * s["d_losses"][1] / s["seq_tokens"][-1].clamp(min=1)
        extra = p * (g - (p * g).sum(1, keepdim=True) + z)
    else:
        extra = p * (1 - score) * (g - (p * g).sum(1, keepdim=True))
    return (out + torch.where(inside, extra, 0.0)).to(s["logits"].dtype)


def _live(s):
    """For each row of the expand buffer its expert, and whether it is a real row."""
    row = torch.arange(s["cap"], device=s["counts"].device)
    offsets, counts = s["offsets"].long(), s["counts"].long()
    expert = torch.searchsorted(offsets[1:], row, right=True).clamp(max=counts.numel() - 1)
    return expert, row - offsets[expert] < counts[expert]


def _plain(s, case):
    op = case["op"]
    if op == "router":
        return _plain_router(s, case)
    if op == "router_backward":
        return _plain_backward(s, case)
    expert, live = _live(s)
    if op == "quantized_matmul":
        E, most = case["E"], s["most"]
        place = (torch.arange(s["cap"], device=live.device) - s["offsets"].long()[expert])[live]
        rows = torch.zeros(E, most, case["in"], device=live.device)
        rows[expert[live], place] = s["x"][live].float()
        y = torch.bmm(rows, s["w"].float().transpose(1, 2))[expert[live], place]
        out = s["y"].clone()  # rows behind an expert's last are left as they were
        out[live] = (y * s["x_scales"][live] * s["w_scales"][expert[live]]).to(out.dtype)
        return out
    v = s["x"].float()
    if op == "swiglu_quantize":
        gate, up = v.split(case["width"], 1)
        v = gate / (1 + torch.exp(-gate)) * up
    top = v.abs().amax(1, keepdim=True).clamp(min=LEAST)
    # the product of two 32-bit numbers is exact in 64, so that a value between two codes goes to the even one
    code = torch.round(v.double() * (torch.full_like(top, 127.0) / top).double())
    codes = torch.where(live[:, None], code.to(torch.int8), s["codes"])
    scales = torch.where(live[:, None], (top / 127).expand(-1, case["copies"]), s["scales"])
    return {"codes": codes.to(torch.bfloat16) if op == "swiglu_quantize" else codes, "scales": scales}


def _own(s, case):
    from combine_ep_layout_amd import binding as B
    op, stream = case["op"], torch.cuda.current_stream()
    kinds = {"bf16": B.EP_BF16, "fp32": B.EP_FP32}
    if op in ("router", "router_backward"):
        kind, S = kinds[case["rows"]], case["S"]
        softmax = case["scoring"] == "softmax"
        shape = (case["T"], case["E"], case["K"], max(S, 1), kind, B.EP_SOFTMAX if softmax else B.EP_SIGMOID,
                 int(case["normalize"]), s["scale"])
        if op == "router_backward":
            B.ep_router_backward(s["logits"], s["idx"], s["seq_offsets"], s["counts"], s["seq_tokens"], s["d_weights"],
                                 s["d_losses"], s["d_losses"][1:] if softmax else None, *shape, s["d_logits"], stream)
            return s["d_logits"]
        loss = s["losses"] if S else None
        B.ep_router(s["logits"], s["bias"], s["mask"], s["seq_offsets"], *shape, int(case["given"]), s["idx"], s["weights"],
                    s["counts"] if S else None, s["seq_tokens"] if S else None, loss, loss[1:] if S and softmax else None,
                    s["workspace"], s["workspace"].numel(), stream)
        out = {"idx": s["idx"], "weights": s["weights"]}
        if S:
            out.update(counts=s["counts"], seq_tokens=s["seq_tokens"], losses=loss if softmax else loss[:1])
        return out
    if op == "quantized_matmul":
        B.ep_quantized_matmul(s["x"], s["x_scales"], 1, s["w"], s["w_scales"], s["counts"], s["offsets"], case["E"], s["cap"],
                              case["in"], case["out"], s["y"], kinds[case["y"]], stream)
        return s["y"]
    call = B.ep_quantize_rows if op == "quantize_rows" else B.ep_swiglu_quantize
    call(s["x"], s["counts"], s["offsets"], case["E"], s["cap"], case["width"], kinds[case["rows"]], s["codes"], s["scales"],
         case["copies"], stream)
    # a rounding between two codes may go either way where the activation itself is rounded: codes as the values they are
    return {"codes": s["codes"].to(torch.bfloat16) if op == "swiglu_quantize" else s["codes"], "scales": s["scales"]}


def run(state):
    return _own(state, state["case"]) if own else _plain(state, state["case"])


# ---------------------------------------------------------------------------------------- work

def _active(case):
    """Experts that get a token, on the average."""
    T, K, E = case["T"], case["K"], case["E"]
    if case["routing"] == "uniform":
        return E * (1 - (1 - K / E) ** T)
    gen = torch.Generator().manual_seed(7)
    noise = torch.rand(min(T, 4096), E, generator=gen, dtype=torch.float64).clamp_(1e-12, 1 - 1e-12)
    key = -1.1 * torch.log1p(torch.arange(E, dtype=torch.float64)) - torch.log(-torch.log(noise))
    return int(torch.unique(key.argsort(dim=1, descending=True)[:, :K]).numel())


def work(case):
    op, T, K, E = (case[k] for k in ("op", "T", "K", "E"))
    e = 2 if case.get("rows") == "bf16" else 4
    if op in ("router", "router_backward"):
        S = case["S"]
        seen = S * (4 * E + 8) if S else 0
        moved = e * T * E * (1 if op == "router" else 2) + 8 * T * K
        return {"bytes": moved + seen, "flops": T * E * (10 if op == "router" else 14)}
    n, routing = T * K, 8 * E + 4
    if op == "quantized_matmul":
        C, N = case["in"], case["out"]
        return {"bytes": _active(case) * N * (C + 4) + n * (C + 4 + N * (2 if case["y"] == "bf16" else 4)) + routing,
                "flops": 2 * n * N * C}
    W = case["width"]
    if op == "quantize_rows":
        return {"bytes": n * (W * e + W + 4 * case["copies"]) + routing, "flops": 3 * n * W}
    return {"bytes": n * (2 * W * e + W + 4 * case["copies"]) + routing, "flops": 9 * n * W}


# ---------------------------------------------------------------------------------------- definition in 64 bits

def _router_terms(l, ids, s, case):
    """(weights, balance loss, z loss) of logits in 64 bits, differentiable."""
    T, E, K, S = case["T"], case["E"], case["K"], max(case["S"], 1)
    p = torch.softmax(l, 1)
    score = p if case["scoring"] == "softmax" else torch.sigmoid(l)
    if case["scoring"] == "sigmoid":
        p = score / score.sum(1, keepdim=True)
    here = ids >= 0
    w = score.gather(1, ids.clamp(min=0)) * here
    if case["normalize"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total > 0, total, torch.ones_like(total))
    bounds = [0, T] if s["seq_offsets"] is None else s["seq_offsets"].tolist()
    parts, counts, tokens = [], [], []
    for b, end in zip(bounds[:-1], bounds[1:]):
        i, on = ids[b:end], here[b:end].any(1)
        c = torch.bincount(i[i >= 0], minlength=E)
        n = int(on.sum())
        counts.append(c)
        tokens.append(n)
        if n:
            parts.append((c.double() * E / (K * n) * p[b:end][on].mean(0)).sum())
    zero = torch.zeros((), dtype=torch.float64, device=l.device)
    balance = torch.stack(parts).mean() if parts else zero
    z = zero
    if case["scoring"] == "softmax" and sum(tokens):
        on = here.any(1)
        on[:bounds[0]] = False
        on[bounds[-1]:] = False
        z = (torch.logsumexp(l[on], 1) ** 2).mean()
    tokens += [sum(n > 0 for n in tokens), sum(tokens)]
    return w * s["scale"], balance, z, torch.stack(counts), torch.tensor(tokens)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "router":
        l = s["logits"].double()
        ids = s["idx"].long()
        if not case["given"]:
            score = torch.sigmoid(l) if case["scoring"] == "sigmoid" else torch.softmax(l, 1)
            key = l if s["bias"] is None else torch.where(torch.isinf(l), l, score + s["bias"].double())
            v, ids = key.sort(dim=1, descending=True, stable=True)
            ids = ids[:, :case["K"]].masked_fill(v[:, :case["K"]] == -math.inf, -1)
            if s["mask"] is not None:
                ids = ids.masked_fill(s["mask"][:, None] == 0, -1)
        w, balance, z, counts, tokens = _router_terms(l, ids, s, case)
        out = {"idx": ids.int(), "weights": w}
        if case["S"]:
            losses = [balance, z] if case["scoring"] == "softmax" else [balance]
            out.update(counts=counts.int(), seq_tokens=tokens.int(), losses=torch.stack(losses))
        return out
    if op == "router_backward":
        l = s["logits"].double().requires_grad_()
        w, balance, z, _, _ = _router_terms(l, s["idx"].long(), s, case)
        total = (w * s["d_weights"].double()).sum() + balance * s["d_losses"][0].double() + z * s["d_losses"][1].double()
        return torch.autograd.grad(total, l)[0]
    begin, count = s["offsets"].tolist(), s["counts"].tolist()
    spans = [(e, slice(begin[e], begin[e] + count[e])) for e in range(case["E"])]
    if op == "quantized_matmul":
        y = torch.zeros(s["cap"], case["out"], dtype=torch.float64, device="cuda")
        for e, r in spans:
            if r.stop > r.start:
                y[r] = (s["x"][r].double() @ s["w"][e].double().T) * s["x_scales"][r].double() * s["w_scales"][e].double()
        return y
    at = torch.cat([torch.arange(r.start, r.stop, device="cuda") for _, r in spans])
    v = s["x"][at].double()
    if op == "swiglu_quantize":
        gate, up = v.chunk(2, 1)
        v = gate * torch.sigmoid(gate) * up
    top = v.abs().amax(1, keepdim=True).clamp(min=LEAST)
    if op == "quantize_rows":  # by the factor 127 / top in 32 bits, as the operator is defined
        code = torch.round(v * (torch.full_like(top, 127.0) / top).float().double()).to(torch.int8)
    else:
        code = torch.round(v * 127 / top)
    codes = torch.zeros(s["cap"], case["width"], dtype=code.dtype, device="cuda")
    codes[at] = code
    scales = torch.zeros(s["cap"], case["copies"], dtype=torch.float64, device="cuda")
    scales[at] = (top / 127).expand(-1, case["copies"])
    return {"codes": codes, "scales": scales}
