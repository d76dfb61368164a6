"""Cases of the experts' operators: what a call of each takes, its plain form and its definition in 64 bits.

ep_moe_layer        the whole expert layer of a few tokens (decode)
ep_expert_matvec    per-expert matrix-vector products on the expand layout, 4-bit (8-bit, bf16) weights
ep_swiglu           the experts' activation, with an 8-bit checkpoint of its input
ep_swiglu_backward  its backward pass from that checkpoint
ep_expert_wgrad     the experts' weight gradient from 8-bit (or bf16) rows

Rows of expert e are [offsets[e], offsets[e] + counts[e]) of an expand buffer; weights in 8 and 4 bits
carry one fp32 scale per 128 values of a row; a 4-bit byte holds the value of even index in its low half.
"""
import math

import numpy as np
import torch

own = False

GROUP = 128
ELT = {"bf16": 2.0, "fp8": 1.0 + 4 / GROUP, "fp4": 0.5 + 4 / GROUP}  # bytes per weight, scales included
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    layer, mv = {"op": "moe_layer"}, {"op": "expert_matvec"}
    fwd, bwd, wg = {"op": "swiglu"}, {"op": "swiglu_backward"}, {"op": "expert_wgrad"}
    return [
        # one token of one sequence: eight experts' weights are all there is to read
        {"name": "layer_one_token_bf16", **layer, "T": 1, "K": 8, "E": 64, "H": 7168, "I": 2048, "weights": "bf16",
         "routing": "uniform", "masked": 0.0, "bias": False},
        # a few sequences on a small model: latency counts; some entries masked, a residual row added
        {"name": "layer_few_tokens_fp8", **layer, "T": 7, "K": 4, "E": 32, "H": 2048, "I": 768, "weights": "fp8",
         "routing": "uniform", "masked": 0.1, "bias": True},
        # the decode batch of 128 tokens over 256 experts with skewed popularity
        {"name": "layer_decode_zipf_fp4", **layer, "T": 128, "K": 8, "E": 256, "H": 7168, "I": 2048,
         "weights": "fp4", "routing": "zipf", "masked": 0.0, "bias": False},
        # one dense projection of one token (a shared expert)
        {"name": "matvec_one_row_fp4", **mv, "T": 1, "K": 1, "E": 1, "A": 1, "in": 7168, "out": 4096,
         "weights": "fp4", "routing": "uniform"},
        # the up projection of a decode batch, expert-major
        {"name": "matvec_decode_fp4", **mv, "T": 128, "K": 8, "E": 64, "A": 1, "in": 7168, "out": 4096,
         "weights": "fp4", "routing": "uniform"},
        # activation of a small odd batch
        {"name": "swiglu_small_bf16", **fwd, "T": 61, "K": 6, "E": 64, "A": 1, "I": 1408, "rows": "bf16",
         "routing": "zipf"},
        # activation of the prefill batch: 32768 rows among alignment padding
        {"name": "swiglu_prefill_bf16", **fwd, "T": 4096, "K": 8, "E": 256, "A": 128, "I": 2048, "rows": "bf16",
         "routing": "uniform"},
        # backward of a fine-tuning batch in fp32
        {"name": "swiglu_back_small_fp32", **bwd, "T": 500, "K": 6, "E": 64, "A": 16, "I": 1408, "rows": "fp32",
         "routing": "zipf"},
        # backward of the prefill-sized training batch
        {"name": "swiglu_back_prefill_bf16", **bwd, "T": 4096, "K": 8, "E": 256, "A": 128, "I": 2048,
         "rows": "bf16", "routing": "uniform"},
        # 128 rows per expert from 8-bit rows as dispatch moves them: the gradient itself is what is written
        {"name": "wgrad_many_experts_fp8", **wg, "T": 1024, "K": 8, "E": 64, "A": 1, "in": 7168, "out": 4096,
         "rows": "fp8", "grad": "bf16", "previous": False, "routing": "uniform"},
        # few experts with thousands of rows each, added to a running fp32 gradient
        {"name": "wgrad_few_experts_bf16", **wg, "T": 8192, "K": 2, "E": 8, "A": 128, "in": 4096, "out": 2048,
         "rows": "bf16", "grad": "fp32", "previous": True, "routing": "uniform"},
        # a small odd batch; some experts get no row
        {"name": "wgrad_small_bf16", **wg, "T": 61, "K": 2, "E": 16, "A": 1, "in": 256, "out": 520,
         "rows": "bf16", "grad": "bf16", "previous": False, "routing": "zipf"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["moe_layer", "expert_matvec", "swiglu", "swiglu_backward", "expert_wgrad"])
    E = _log_int(rng, 1, 256)
    K = min(E, rng.choice([1, 2, 4, 6, 8]))
    case = {"op": op, "K": K, "E": E, "routing": rng.choice(["uniform", "zipf"])}
    if op in ("moe_layer", "expert_matvec"):
        weights = rng.choice(["bf16", "fp8", "fp4"])
        step = 8 if weights == "bf16" else GROUP
        wide = _log_int(rng, 256, 7168 if E <= 64 else 2048) // step * step
        narrow = _log_int(rng, 128, 2048) // step * step
        T = _log_int(rng, 1, 128)
        if op == "moe_layer":
            return {**case, "T": T, "H": wide, "I": narrow, "weights": weights,
                    "masked": rng.choice([0.0, 0.3]), "bias": rng.random() < 0.5}
        return {**case, "T": T, "A": rng.choice([1, 16]), "in": wide, "out": _log_int(rng, 64, 4096) // 8 * 8,
                "weights": weights}
    if op in ("swiglu", "swiglu_backward"):
        return {**case, "T": _log_int(rng, 1, 2048), "A": rng.choice([1, 16, 128]), "I": GROUP * _log_int(rng, 1, 16),
                "rows": rng.choice(["bf16", "fp32"])}
    rows = rng.choice(["fp8", "bf16"])
    return {**case, "E": min(E, 32), "K": min(K, 2, E), "T": _log_int(rng, 1, 4096), "A": rng.choice([1, 16, 128]),
            "in": _log_int(rng, 1, 32) * GROUP if rows == "fp8" else _log_int(rng, 64, 4096) // 8 * 8,
            "out": _log_int(rng, 64, 2048) // 8 * 8, "rows": rows, "grad": rng.choice(["bf16", "fp32"]),
            "previous": rng.random() < 0.5}


# ---------------------------------------------------------------------------------------- inputs

def _zipf(noise, order):
    """K distinct experts a token from a Zipf(1.1) popularity: the largest of log-popularity + Gumbel noise."""
    return (-1.1 * torch.log1p(order.double()))[None, :] - torch.log(-torch.log(noise))


def _route(case, gen):
    noise = torch.rand(case["T"], case["E"], generator=gen, device=gen.device, dtype=torch.float64).clamp_(1e-12, 1 - 1e-12)
    if case["routing"] == "zipf":
        noise = _zipf(noise, torch.randperm(case["E"], generator=gen, device=gen.device))
    return noise.argsort(dim=1, descending=True)[:, :case["K"]].to(torch.int32).contiguous()


def _weights(shape, kind, gen):
    """A weight matrix per expert of entries about 1/sqrt(width), and its scales."""
    E, N, C = shape
    std = C ** -0.5
    if kind == "bf16":
        w = torch.empty(shape, dtype=torch.bfloat16, device="cuda")
        w.normal_(0.0, std, generator=gen)
        return w, None
    scales = torch.empty(E, N, C // GROUP, device="cuda").uniform_(0.7, 1.4, generator=gen)
    if kind == "fp8":  # normal values over a range of e4m3, whose scale brings them back
        w = torch.empty(shape, dtype=torch.float8_e4m3fn, device="cuda")
        for e in range(E):
            w[e] = torch.empty(N, C, device="cuda").normal_(0.0, 100.0, generator=gen).clamp_(-448, 448).to(w.dtype)
        return w.view(torch.uint8), scales.mul_(std / 100.0)
    w = torch.empty(E, N, C // 2, dtype=torch.uint8, device="cuda")
    edges = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    v = torch.empty(1 << 20, 2, device="cuda").normal_(0.0, 2.0, generator=gen)
    code = torch.bucketize(v.abs(), edges) + 8 * (v < 0)
    pairs = (code[:, 0] + 16 * code[:, 1]).to(torch.uint8)  # bytes as rounding normal values leaves them
    for e in range(E):
        w[e] = pairs[torch.randint(0, 1 << 20, (N, C // 2), generator=gen, device="cuda")]
    return w, scales.mul_(std / 2.0)


def _expand(case, gen):
    """The routing arrays of an expand buffer: counts, offsets and the buffer's rows."""
    T, K, E, A = (case[k] for k in ("T", "K", "E", "A"))
    idx = _route(case, gen).reshape(-1).long()
    counts = torch.bincount(idx, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int64, device="cuda")
    offsets[1:] = torch.cumsum((counts + A - 1) // A * A, 0)
    return counts.to(torch.int32), offsets.to(torch.int32), T * K + E * (A - 1), int(counts.max())


def _checkpoint(v):
    """e4m3 codes of rows and one power-of-two scale per 128 values: the smallest that keeps them within 448."""
    g = v.float().unflatten(-1, (-1, GROUP))
    m, e = torch.frexp(g.abs().amax(-1))
    s = torch.ldexp(torch.ones_like(m), torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126))
    return (g / s[..., None]).to(torch.float8_e4m3fn).flatten(-2), s


def _rows(n, width, kind, gen, std):
    return torch.empty(n, width, dtype=torch.float32 if kind == "fp32" else torch.bfloat16, device="cuda").normal_(0.0, std, generator=gen)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    s = {"case": case}
    if op == "moe_layer":
        T, K, E, H, I = (case[k] for k in ("T", "K", "E", "H", "I"))
        idx = _route(case, gen)
        idx[torch.rand(T, K, generator=gen, device="cuda") < case["masked"]] = -1
        s["idx"] = idx
        s["probs"] = torch.softmax(torch.randn(T, K, generator=gen, device="cuda"), dim=1)
        s["x"] = _rows(T, H, "bf16", gen, 1.0)
        s["bias"] = _rows(T, H, "bf16", gen, 0.5) if case["bias"] else None
        s["w_in"], s["in_scales"] = _weights((E, 2 * I, H), case["weights"], gen)
        s["w_out"], s["out_scales"] = _weights((E, H, I), case["weights"], gen)
        s["out"] = torch.empty(T, H, dtype=torch.bfloat16, device="cuda")
        s["workspace"] = torch.empty(T * K * (4 * I + 16) + 4096, dtype=torch.uint8, device="cuda")
        return s
    s["counts"], s["offsets"], s["cap"], s["most"] = _expand(case, gen)
    cap = s["cap"]
    if op == "expert_matvec":
        s["x"] = _rows(cap, case["in"], "bf16", gen, 1.0)
        s["w"], s["scales"] = _weights((case["E"], case["out"], case["in"]), case["weights"], gen)
        s["y"] = torch.zeros(cap, case["out"], dtype=torch.bfloat16, device="cuda")
    elif op == "swiglu":
        I, kind = case["I"], case["rows"]
        s["gate_up"] = _rows(cap, 2 * I, kind, gen, 1.5)
        s["h"] = torch.zeros(cap, I, dtype=s["gate_up"].dtype, device="cuda")
        s["codes"] = torch.zeros(cap, 2 * I, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.zeros(cap, 2 * I // GROUP, device="cuda")
    elif op == "swiglu_backward":
        I, kind = case["I"], case["rows"]
        codes, s["scales"] = _checkpoint(_rows(cap, 2 * I, "fp32", gen, 1.5))
        s["codes"] = codes.view(torch.uint8)
        s["dh"] = _rows(cap, I, kind, gen, 1e-2)
        s["h"] = torch.zeros_like(s["dh"])
        s["d_gate_up"] = torch.zeros(cap, 2 * I, dtype=s["dh"].dtype, device="cuda")
    else:
        E, N, C = case["E"], case["out"], case["in"]
        s["dy"] = _rows(cap, N, "bf16", gen, 1e-2)
        if case["rows"] == "fp8":
            codes, s["scales"] = _checkpoint(_rows(cap, C, "fp32", gen, 1.0))
            s["x"] = codes.view(torch.uint8)
        else:
            s["x"], s["scales"] = _rows(cap, C, "bf16", gen, 1.0), None
        kind = torch.float32 if case["grad"] == "fp32" else torch.bfloat16
        s["previous"] = torch.empty(E, N, C, dtype=kind, device="cuda").normal_(0.0, 0.05, generator=gen) if case["previous"] else None
        s["dw"] = torch.empty(E, N, C, dtype=kind, device="cuda")
    return s


# ---------------------------------------------------------------------------------------- plain forms

def _values(w, scales, kind):
    """Weights or rows as the values they stand for, in 32 bits."""
    if kind == "bf16":
        return w.float()
    if kind == "fp8":
        v = w.view(torch.float8_e4m3fn).float()
    else:
        half = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=w.device)
        byte = torch.arange(256, device=w.device)
        both = torch.stack([half[byte % 16], half[byte // 16]], 1)
        v = both.index_select(0, w.reshape(-1).int()).view(*w.shape[:-1], -1)
    v.unflatten(-1, (-1, GROUP)).mul_(scales[..., None])
    return v


def _products(x, expert, w, scales, kind, most):
    """y[i] = W[expert[i]] x[i] in 32 bits. Fewer rows than experts: each row's own matrix; else the rows of
    each expert side by side."""
    n, E = expert.numel(), w.shape[0]
    if n < E:
        return torch.bmm(_values(w[expert], None if scales is None else scales[expert], kind), x[:, :, None])[:, :, 0]
    hit = torch.nn.functional.one_hot(expert, E)
    place = (hit.cumsum(0) - hit).gather(1, expert[:, None])[:, 0].clamp(max=most)  # beyond `most`: rows whose result is not used
    rows = torch.zeros(E, most + 1, x.shape[1], device=x.device)
    rows[expert, place] = x
    return torch.bmm(rows, _values(w, scales, kind).transpose(1, 2))[expert, place]


def _live(s):
    """For each row of the expand buffer its expert, and whether it is a real row."""
    row = torch.arange(s["cap"], device=s["counts"].device)
    offsets, counts = s["offsets"].long(), s["counts"].long()
    expert = torch.searchsorted(offsets[1:], row, right=True).clamp(max=counts.numel() - 1)
    return expert, row - offsets[expert] < counts[expert]


def _plain_layer(s, case):
    T, K, I = case["T"], case["K"], case["I"]
    idx = s["idx"].reshape(-1).long()
    valid = idx >= 0
    expert = idx.clamp(min=0)
    # a masked entry is counted with expert 0, so that expert may hold every entry
    most = T if case["masked"] == 0 else T * K
    x = s["x"].float().repeat_interleave(K, 0)
    gate, up = _products(x, expert, s["w_in"], s["in_scales"], case["weights"], most).split(I, 1)
    h = gate / (1 + torch.exp(-gate)) * up
    y = _products(h, expert, s["w_out"], s["out_scales"], case["weights"], most)
    y = torch.where(valid[:, None], y * s["probs"].reshape(-1, 1), torch.zeros_like(y)).view(T, K, -1).sum(1)
    return (y if s["bias"] is None else y + s["bias"].float()).to(torch.bfloat16)


def _plain(s, case):
    op = case["op"]
    if op == "moe_layer":
        return _plain_layer(s, case)
    expert, live = _live(s)
    if op == "expert_matvec":
        # rows behind an expert's last are left as they were
        at = torch.nonzero(live)[:, 0]
        y = s["y"].clone()
        y[at] = _products(s["x"][at].float(), expert[at], s["w"], s["scales"], case["weights"], s["most"]).to(y.dtype)
        return y
    live = live[:, None]
    if op == "swiglu":
        I = case["I"]
        v = s["gate_up"].float()
        gate, up = v.split(I, 1)
        h = gate / (1 + torch.exp(-gate)) * up
        codes, scales = _checkpoint(v)
        return {"h": torch.where(live, h.to(s["h"].dtype), s["h"]),
                "checkpoint": torch.where(live, codes.view(torch.uint8), s["codes"]).view(torch.float8_e4m3fn),
                "scales": torch.where(live, scales, s["scales"])}
    if op == "swiglu_backward":
        gate, up = _values(s["codes"], s["scales"], "fp8").split(case["I"], 1)
        dh = s["dh"].float()
        sig = 1 / (1 + torch.exp(-gate))
        d = torch.cat([dh * up * sig * (1 + gate * (1 - sig)), dh * gate * sig], 1)
        kind = s["dh"].dtype
        return {"d_gate_up": torch.where(live, d.to(kind), s["d_gate_up"]),
                "h": torch.where(live, (gate * sig * up).to(kind), s["h"])}
    at = s["offsets"][:-1, None].long() + torch.arange(s["most"], device=expert.device)  # [E, most]
    real = (torch.arange(s["most"], device=expert.device) < s["counts"][:, None])[..., None]
    at = at.clamp(max=max(s["cap"] - 1, 0))
    dy = torch.where(real, s["dy"][at].float(), 0.0)
    x = torch.where(real, _values(s["x"][at], None if s["scales"] is None else s["scales"][at], case["rows"]), 0.0)
    dw = torch.bmm(dy.transpose(1, 2), x)
    return (dw if s["previous"] is None else dw + s["previous"].float()).to(s["dw"].dtype)


def _own(s, case):
    from combine_ep_layout_amd import binding as B
    op, stream = case["op"], torch.cuda.current_stream()
    kinds = {"bf16": B.EP_BF16, "fp32": B.EP_FP32, "fp8": B.EP_FP8_E4M3, "fp4": B.EP_FP4X2}
    if op == "moe_layer":
        B.ep_moe_layer(s["x"], s["idx"], s["probs"], s["bias"], s["w_in"], s["in_scales"], s["w_out"], s["out_scales"],
                       case["T"], case["H"], case["I"], case["K"], case["E"], kinds[case["weights"]], s["out"],
                       s["workspace"], s["workspace"].numel(), stream)
        return s["out"]
    if op == "expert_matvec":
        B.ep_expert_matvec(s["x"], s["w"], s["scales"], s["counts"], s["offsets"], case["E"], s["cap"], case["in"],
                           case["out"], kinds[case["weights"]], s["y"], B.EP_BF16, stream)
        return s["y"]
    if op == "swiglu":
        B.ep_swiglu(s["gate_up"], s["counts"], s["offsets"], case["E"], s["cap"], case["I"], kinds[case["rows"]], s["h"],
                    s["codes"], s["scales"], stream)
        return {"h": s["h"], "checkpoint": s["codes"].view(torch.float8_e4m3fn), "scales": s["scales"]}
    if op == "swiglu_backward":
        B.ep_swiglu_backward(s["dh"], s["codes"], s["scales"], s["counts"], s["offsets"], case["E"], s["cap"], case["I"],
                             kinds[case["rows"]], s["d_gate_up"], s["h"], stream)
        return {"d_gate_up": s["d_gate_up"], "h": s["h"]}
    B.ep_expert_wgrad(s["dy"], s["x"], s["scales"], s["counts"], s["offsets"], case["E"], s["cap"], case["out"], case["in"],
                      kinds[case["rows"]], s["previous"], s["dw"], kinds[case["grad"]], stream)
    return s["dw"]


def run(state):
    return _own(state, state["case"]) if own else _plain(state, state["case"])


# ---------------------------------------------------------------------------------------- work

def _active(case):
    """Experts that get a token, on the average (skewed routing: of a few seeded draws)."""
    T, K, E = case["T"], case["K"], case["E"]
    if case["routing"] == "uniform":
        return E * (1 - (1 - K / E) ** T)
    rng = np.random.default_rng(7)
    p = -1.1 * np.log(np.arange(1, E + 1)) + rng.gumbel(size=(4, T, E))
    top = np.argsort(-p, axis=2)[:, :, :K]
    return sum(len(np.unique(t)) for t in top) / 4


def work(case):
    op, T, K, E = (case[k] for k in ("op", "T", "K", "E"))
    n = T * K
    if op == "moe_layer":
        H, I = case["H"], case["I"]
        kept = n * (1 - case["masked"])
        weights = _active({**case, "K": max(K * (1 - case["masked"]), 1) if case["routing"] == "uniform" else K}) * 3 * I * H
        return {"bytes": weights * ELT[case["weights"]] + T * H * (6 if case["bias"] else 4) + 8 * n, "flops": 6 * kept * I * H}
    routing = 8 * E + 4
    if op == "expert_matvec":
        N, C = case["out"], case["in"]
        return {"bytes": _active(case) * N * C * ELT[case["weights"]] + 2 * n * (N + C) + routing, "flops": 2 * n * N * C}
    if op in ("swiglu", "swiglu_backward"):
        I, e = case["I"], 4 if case["rows"] == "fp32" else 2
        kept = 2 * I * (1 + 4 / GROUP)
        moved = 3 * I * e if op == "swiglu" else 4 * I * e
        return {"bytes": n * (moved + kept) + routing, "flops": n * I * (12 if op == "swiglu" else 18)}
    N, C, g = case["out"], case["in"], 4 if case["grad"] == "fp32" else 2
    return {"bytes": n * (2 * N + C * ELT[case["rows"]]) + E * N * C * g * (2 if case["previous"] else 1) + routing,
            "flops": 2 * n * N * C}


# ---------------------------------------------------------------------------------------- definition in 64 bits

def _double(w, scales, kind):
    """One matrix of weights or rows in 64 bits."""
    if kind == "fp4":
        code = torch.stack([w & 15, w >> 4], -1).flatten(-2).long()
        v = torch.tensor(E2M1, dtype=torch.float64, device=w.device)[code & 7] * (1 - 2 * (code >> 3)).double()
    else:
        v = (w.view(torch.float8_e4m3fn) if kind == "fp8" else w).double()
    return v if scales is None else v * scales.double().repeat_interleave(GROUP, -1)


def _at(scales, e):
    return None if scales is None else scales[e]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "moe_layer":
        out = torch.zeros(case["T"], case["H"], dtype=torch.float64, device="cuda")
        for e in torch.unique(s["idx"]).tolist():
            if e < 0:
                continue
            t, k = torch.nonzero(s["idx"] == e, as_tuple=True)
            z = s["x"][t].double() @ _double(s["w_in"][e], _at(s["in_scales"], e), case["weights"]).T
            gate, up = z[:, :case["I"]], z[:, case["I"]:]
            y = (gate * torch.sigmoid(gate) * up) @ _double(s["w_out"][e], _at(s["out_scales"], e), case["weights"]).T
            out.index_add_(0, t, y * s["probs"][t, k].double()[:, None])
        return out if s["bias"] is None else out + s["bias"].double()
    begin, count = s["offsets"].tolist(), s["counts"].tolist()
    spans = [(e, slice(begin[e], begin[e] + count[e])) for e in range(case["E"])]
    if op == "expert_matvec":
        y = torch.zeros(s["cap"], case["out"], dtype=torch.float64, device="cuda")
        for e, r in spans:
            if r.stop > r.start:
                y[r] = s["x"][r].double() @ _double(s["w"][e], _at(s["scales"], e), case["weights"]).T
        return y
    if op == "expert_wgrad":
        dw = torch.zeros(case["E"], case["out"], case["in"], dtype=torch.float64, device="cuda")
        for e, r in spans:
            dw[e] = s["dy"][r].double().T @ _double(s["x"][r], None if s["scales"] is None else s["scales"][r], case["rows"])
        return dw if s["previous"] is None else dw + s["previous"].double()
    at = torch.cat([torch.arange(r.start, r.stop, device="cuda") for _, r in spans])
    I = case["I"]
    if op == "swiglu":
        v = s["gate_up"][at].double()
        h = torch.zeros(s["cap"], I, dtype=torch.float64, device="cuda")
        h[at] = v[:, :I] * torch.sigmoid(v[:, :I]) * v[:, I:]
        # the checkpoint's codes and scales: the smallest power of two that keeps 128 values within 448
        group = v.unflatten(1, (-1, GROUP))
        power = torch.ceil(torch.log2(group.abs().amax(-1) / 448)).clamp(min=-126)
        codes = torch.zeros(s["cap"], 2 * I, dtype=torch.float64, device="cuda")
        codes[at] = (group / torch.exp2(power)[..., None]).flatten(1).float().to(torch.float8_e4m3fn).double()
        scales = torch.zeros(s["cap"], 2 * I // GROUP, dtype=torch.float64, device="cuda")
        scales[at] = torch.exp2(power)
        return {"h": h, "checkpoint": codes, "scales": scales}
    v = _double(s["codes"][at], s["scales"][at], "fp8")
    gate, up, dh = v[:, :I], v[:, I:], s["dh"][at].double()
    sig = torch.sigmoid(gate)
    d = torch.zeros(s["cap"], 2 * I, dtype=torch.float64, device="cuda")
    h = torch.zeros(s["cap"], I, dtype=torch.float64, device="cuda")
    d[at] = torch.cat([dh * up * sig * (1 + gate * (1 - sig)), dh * gate * sig], 1)
    h[at] = gate * sig * up
    return {"d_gate_up": d, "h": h}
