"""The router's operators on the GPU against plain 64-bit forms (tests/router_ref.py).

Ids, counts and numbers of tokens have to be equal; weights, losses and gradients lie within bounds
derived there. Shapes sit where the kernels can go wrong: one token, one expert, expert numbers around
the lanes' and loads' widths, top-k up to 64, tied and nearly tied keys, masked tokens, experts at
-infinity or the type's lowest value, rows with nothing left, ids given twice or outside, sequences
that are empty, end inside a tile or leave tokens out, workgroup caps, other streams, graph replays.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - only on CPU hosts
    pytest.skip("needs a GPU", allow_module_level=True)

from combine_ep_layout_amd import binding as B  # noqa: E402
from tests import router_ref as R  # noqa: E402

DEV = "cuda:0"
KIND = {"bf16": B.EP_BF16, "fp32": B.EP_FP32}
TYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}
SCORING = {"softmax": B.EP_SOFTMAX, "sigmoid": B.EP_SIGMOID}
INF = float("inf")


def _say(msg):
    print(msg, flush=True)


def _gen(*seed):
    n = 0
    for s in seed:
        n = n * 1000003 + int(s)
    return torch.Generator(device=DEV).manual_seed(n % (1 << 62))


def _ints(shape):
    return torch.full(shape, -7, dtype=torch.int32, device=DEV)


class Forward:
    """A forward call's operands, and the call."""

    def __init__(self, logits, K, scoring, normalize=True, scale=1.0, bias=None, mask=None, seq=None, ids=None, stats=True):
        self.l, self.K, self.scoring, self.normalize, self.scale = logits, K, scoring, normalize, scale
        self.T, self.E = logits.shape
        self.bias, self.mask, self.seq, self.given, self.stats = bias, mask, seq, ids is not None, stats
        self.S = 1 if seq is None else seq.numel() - 1
        self.kind = "fp32" if logits.dtype == torch.float32 else "bf16"
        self.idx = ids.to(torch.int32).clone() if self.given else _ints((self.T, K))
        self.w = torch.full((self.T, K), -7.0, device=DEV)
        self.counts, self.tokens = (_ints((self.S, self.E)), _ints((self.S + 2,))) if stats else (None, None)
        self.losses = torch.full((2,), -7.0, device=DEV)
        need = B.ep_router_workspace_bytes(self.T, self.E, self.S)
        self.ws = torch.full((need + 64,), 0xA5, dtype=torch.uint8, device=DEV) if stats else None
        self.need = need

    def __call__(self, stream=None):
        soft = self.scoring == "softmax"
        B.ep_router(self.l, self.bias, self.mask, self.seq, self.T, self.E, self.K, self.S, KIND[self.kind], SCORING[self.scoring],
                    int(self.normalize), self.scale, int(self.given), self.idx, self.w, self.counts, self.tokens,
                    self.losses if self.stats else None, self.losses[1:] if self.stats and soft else None, self.ws,
                    self.need if self.stats else 0, stream)
        return self

    def check(self):
        torch.cuda.synchronize()
        l = self.l.double()
        if self.given:
            ids = torch.where((self.idx >= 0) & (self.idx < self.E), self.idx.long(), -1)
        else:
            ids = R.choose(l, self.K, self.scoring, self.bias, self.mask)
            assert torch.equal(self.idx.long(), ids), f"ids differ in rows {torch.nonzero((self.idx != ids).any(1))[:5].flatten().tolist()}"
        self.ids = ids
        w, err = R.weights(l, ids, self.scoring, self.normalize, self.scale)
        R.near(self.w, w, err, torch.float32)
        if self.stats:
            counts, tokens, (balance, db), (z, dz) = R.statistics(l, ids, self.scoring, self.seq)
            assert torch.equal(self.counts.long(), counts) and torch.equal(self.tokens.long(), tokens)
            assert abs(float(self.losses[0]) - balance) <= db + U * abs(balance), (float(self.losses[0]), balance)
            if self.scoring == "softmax":
                assert abs(float(self.losses[1]) - z) <= dz + U * abs(z), (float(self.losses[1]), z)
            else:
                assert float(self.losses[1]) == -7.0
            assert bool((self.ws[self.need:] == 0xA5).all()), "written behind the workspace"
        return self


U = R.U


def _backward(f, dw, db, dz, stream=None, check=True):
    """The backward call of a checked forward one; returns d_logits."""
    d = torch.full_like(f.l, -7.0)
    grads = [None if g is None else torch.full((1,), g, device=DEV) for g in (db, dz)]
    torch.cuda.synchronize()
    B.ep_router_backward(f.l, f.idx, f.seq, f.counts, f.tokens, dw, *grads, f.T, f.E, f.K, f.S, KIND[f.kind], SCORING[f.scoring],
                         int(f.normalize), f.scale, d, stream)
    if check:
        torch.cuda.synchronize()
        as32 = [None if g is None else float(torch.tensor(g)) for g in (db, dz)]
        want, err = R.backward(f.l.double(), f.ids, f.scoring, f.normalize, f.scale, dw, f.seq,
                               f.counts, f.tokens, *as32)
        R.near(d, want, err, f.l.dtype)
    return d


def _logits(T, E, kind, gen, std=1.5):
    return (torch.randn(T, E, generator=gen, device=DEV) * std).to(TYPE[kind])


SHAPES = [
    # T, E, K, kind
    (1, 1, 1, "fp32"), (1, 256, 8, "bf16"), (3, 2, 2, "bf16"), (17, 16, 4, "fp32"), (65, 17, 3, "bf16"), (64, 32, 6, "fp32"),
    (100, 33, 5, "fp32"), (129, 60, 4, "bf16"), (64, 64, 64, "fp32"), (50, 65, 8, "bf16"), (33, 127, 7, "fp32"), (70, 128, 8, "bf16"),
    (257, 160, 6, "fp32"), (1000, 256, 8, "fp32"), (130, 256, 64, "bf16"), (40, 257, 8, "fp32"), (31, 384, 8, "bf16"), (90, 512, 9, "fp32"),
    (21, 513, 8, "bf16"), (75, 1000, 16, "fp32"), (64, 1024, 64, "bf16"), (7, 1023, 1, "fp32"), (3000, 64, 6, "bf16"), (20000, 128, 2, "fp32"),
]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,K,kind", SHAPES)
def test_router_and_backward(T, E, K, kind, scoring):
    for variant in range(4):
        gen = _gen(1, T, E, K, variant)
        normalize, biased, masked, sequences = variant % 2 == 0, variant in (1, 2), variant >= 2, variant in (0, 3)
        _say(f"[router] T={T} E={E} K={K} {kind} {scoring} normalize={normalize} bias={biased} masked={masked} sequences={sequences}")
        l = _logits(T, E, kind, gen)
        if variant == 3:
            l[:, torch.rand(E, generator=gen, device=DEV) < 0.3] = -INF
        bias = torch.randn(E, generator=gen, device=DEV) * 0.1 if biased else None
        mask = (torch.rand(T, generator=gen, device=DEV) > 0.2).to(torch.uint8) if masked else None
        seq = None
        if sequences:
            cut = torch.sort(torch.randint(0, T + 1, (max(1, T // 20),), generator=gen, device=DEV)).values
            seq = torch.cat([cut, cut[-1:]]).to(torch.int32)  # the last one empty, tokens before and behind
        f = Forward(l, K, scoring, normalize, 2.5 if variant else 1.0, bias, mask, seq)()
        f.check()
        dw = torch.randn(T, K, generator=gen, device=DEV)
        _backward(f, dw, 0.7, 0.3 if scoring == "softmax" else None)
    _backward(f, None, None, None)
    _backward(f, dw, None, None)
    _backward(f, None, 1.0, None)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("E,K,kind", [(60, 4, "bf16"), (256, 8, "fp32"), (1024, 33, "fp32"), (5, 40, "bf16")])
def test_given_ids_repeated_and_outside(E, K, kind, normalize, scoring):
    _say(f"[given] E={E} K={K} {kind} {scoring} {normalize}")
    T, gen = 300, _gen(2, E, K)
    ids = torch.randint(-2, E + 2, (T, K), generator=gen, device=DEV)
    ids[5] = -1
    ids[6] = E
    ids[7] = 0  # one id in every place
    ids[8, 0] = 2 ** 31 - 1
    ids[9, 0] = -2 ** 31
    seq = torch.tensor([0, 0, 64, 64, 65, 299, 300], dtype=torch.int32, device=DEV)
    f = Forward(_logits(T, E, kind, gen), K, scoring, normalize, -0.5, seq=seq, ids=ids)()
    f.check()
    assert torch.equal(f.idx.long(), ids), "given ids are not written"
    _backward(f, torch.randn(T, K, generator=gen, device=DEV), 1.3, -0.2 if scoring == "softmax" else None)


def test_ties_go_to_the_lowest_id():
    for E in (7, 64, 256, 700):
        _say(f"[ties] E={E}")
        l = torch.zeros(20, E, device=DEV)
        l[3, E // 2:] = 1.0
        l[4] = torch.arange(E, device=DEV) % 3
        l[5] = -0.0
        l[5, 1] = 0.0  # equal to -0
        for kind in ("bf16", "fp32"):
            for scoring in ("softmax", "sigmoid"):
                Forward(l.to(TYPE[kind]), 5, scoring)().check()
                Forward(l.to(TYPE[kind]), 5, scoring, bias=torch.zeros(E, device=DEV))().check()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_keys_that_binary32_cannot_tell_apart(scoring):
    """Logits a step apart, and scores that differ from score + bias by less than a binary32 step."""
    _say(f"[near ties] {scoring}")
    E, T = 200, 400
    gen = _gen(4)
    base = torch.rand(T, 1, generator=gen, device=DEV) * 2 + 1
    steps = torch.randint(0, 6, (T, E), generator=gen, device=DEV)
    l = (base.view(torch.int32) + steps.to(torch.int32)).view(torch.float32)  # neighbouring numbers
    Forward(l, 8, scoring)().check()
    l = torch.randn(T, E, generator=gen, device=DEV)
    score = R.scores(l.double(), scoring)[0]
    bias = (0.5 - score[0]).float()  # row 0: every key is 0.5 up to rounding
    Forward(l, 8, scoring, bias=bias)().check()
    Forward(l, 8, scoring, bias=1000.0 + bias)().check()
    Forward(l[:1].expand(64, E).contiguous(), 64, scoring, bias=bias)().check()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K", [(12, 8), (40, 8), (256, 8), (256, 13), (600, 8), (600, 40)])
def test_neighbours_around_the_last_place(E, K, scoring):
    """Row n has n keys within a few steps of each other around the K-th place, the rest far away."""
    _say(f"[neighbours] E={E} K={K} {scoring}")
    gen = _gen(6, E, K)
    T = min(E, 70)
    l = torch.randn(T, E, generator=gen, device=DEV)
    for n in range(T):
        at = torch.randperm(E, generator=gen, device=DEV)
        above = max(0, min(K - 1 - n // 2, E - n))
        l[n, at[:above]] += 9.0
        steps = torch.randint(0, 40, (n,), generator=gen, device=DEV).to(torch.int32)
        l[n, at[above:above + n]] = (torch.full((n,), 5.0, device=DEV).view(torch.int32) + steps).view(torch.float32)
    Forward(l, K, scoring)().check()
    Forward(l, K, scoring, bias=torch.zeros(E, device=DEV))().check()
    Forward(l, K, scoring, bias=torch.randint(0, 2, (E,), generator=gen, device=DEV).float())().check()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("E", [40, 256, 600])
def test_extreme_logits(E, kind, scoring):
    _say(f"[extreme] E={E} {kind} {scoring}")
    low = torch.finfo(TYPE[kind]).min
    l = _logits(40, E, kind, _gen(5, E))
    l[1] = -INF                      # nothing left
    l[2, 1:] = -INF                  # one left
    l[3] = low                       # all equal at the type's lowest value
    l[4, 2:] = low
    l[5] = -200.0 - torch.arange(E, device=DEV) % 7      # sigmoids that underflow
    l[6] = -100.0
    l[7] = 80.0
    l[7, 3] = 100.0
    l[8, :E // 2] = -INF
    l[9] = 300.0
    l[10, :] = torch.linspace(-50, 50, E, device=DEV)
    K = 6
    z = scoring == "softmax"
    for normalize in (True, False):
        f = Forward(l, K, scoring, normalize)()
        torch.cuda.synchronize()
        # the z loss of logits at the lowest value is beyond binary32: checked without those rows
        ids = R.choose(l.double(), K, scoring)
        assert torch.equal(f.idx.long(), ids)
        keep = torch.ones(40, dtype=torch.bool, device=DEV)
        keep[3] = False
        g = Forward(l[keep].contiguous(), K, scoring, normalize)().check()
        _backward(g, torch.randn(39, K, generator=_gen(6), device=DEV), 0.5, 0.1 if z else None)
        w, err = R.weights(l.double(), ids, scoring, normalize, 1.0)
        R.near(f.w, w, err, torch.float32)
        given = torch.zeros(40, K, dtype=torch.long, device=DEV)
        given[:, 1:] = torch.randint(0, E, (40, K - 1), generator=_gen(7), device=DEV)
        h = Forward(l[keep].contiguous(), K, scoring, normalize, ids=given[keep])().check()
        _backward(h, torch.randn(39, K, generator=_gen(8), device=DEV), 0.5, 0.1 if z else None)


def test_nan_logits_and_biases_are_not_chosen():
    _say("[nan]")
    l = _logits(10, 100, "fp32", _gen(9))
    l[2, 4] = float("nan")
    l[3] = float("nan")
    bias = torch.zeros(100, device=DEV)
    bias[7], bias[8], bias[9] = float("nan"), -INF, INF
    for b in (None, bias):
        f = Forward(l, 8, "sigmoid", bias=b, stats=False)()
        torch.cuda.synchronize()
        assert torch.equal(f.idx.long(), R.choose(l.double(), 8, "sigmoid", b))
        assert not bool(((f.idx == 4)[2]).any()) and bool((f.idx[3] == -1).all()) and bool((f.w[3] == 0).all())
    rows = [r for r in range(10) if r != 3]
    assert bool((f.idx[rows, 0] == 9).all()) and not bool(((f.idx == 7) | (f.idx == 8)).any())


def test_a_row_with_nan_leaves_the_others_alone():
    l = _logits(64, 256, "fp32", _gen(10))
    want = Forward(l, 8, "softmax")().check()
    broken = l.clone()
    broken[9, 3] = float("nan")
    f = Forward(broken, 8, "softmax")()
    torch.cuda.synchronize()
    keep = torch.arange(64, device=DEV) != 9
    assert torch.equal(f.idx[keep], want.idx[keep]) and torch.equal(f.w[keep], want.w[keep])


def test_no_tokens_and_no_outputs_but_the_needed():
    l = torch.empty(0, 32, device=DEV)
    f = Forward(l, 4, "softmax", seq=torch.zeros(4, dtype=torch.int32, device=DEV))()
    torch.cuda.synchronize()
    assert bool((f.counts == 0).all()) and bool((f.tokens == 0).all()) and bool((f.losses == 0).all())
    l = _logits(50, 32, "fp32", _gen(11))
    idx = _ints((50, 4))
    B.ep_router(l, None, None, None, 50, 32, 4, 1, B.EP_FP32, B.EP_SOFTMAX, 1, 1.0, 0, idx, None)
    torch.cuda.synchronize()
    assert torch.equal(idx.long(), R.choose(l.double(), 4, "softmax"))
    f = Forward(l, 4, "softmax", mask=torch.zeros(50, dtype=torch.uint8, device=DEV))().check()
    assert bool((f.idx == -1).all()) and bool((f.losses == 0).all())
    assert bool((_backward(f, torch.ones(50, 4, device=DEV), 1.0, 1.0) == 0).all())


def test_sequences_of_every_length():
    _say("[sequences]")
    gen = _gen(12)
    T, E = 2500, 48
    ends = torch.cumsum(torch.tensor([0, 1, 0, 2, 63, 64, 65, 1, 1, 300, 0, 900, 256, 400], device=DEV), 0)
    seq = torch.cat([torch.tensor([3], device=DEV), 3 + ends]).to(torch.int32)
    for scoring in ("softmax", "sigmoid"):
        f = Forward(_logits(T, E, "fp32", gen), 3, scoring, seq=seq)().check()
        _backward(f, None, 1.0, None)
    every = torch.arange(T + 1, dtype=torch.int32, device=DEV)  # one token each
    f = Forward(f.l, 3, "softmax", seq=every)().check()
    _backward(f, None, 1.0, 0.5)


def test_offsets_that_are_no_sequences_reach_no_memory_outside():
    gen = _gen(13)
    l = _logits(500, 40, "fp32", gen)
    for seq in ([-5, 700], [400, 100], [2 ** 31 - 1, -2 ** 31, 7, 0, 600], [0, 500, 0, 500]):
        f = Forward(l, 4, "softmax", seq=torch.tensor(seq, dtype=torch.int32, device=DEV))()
        torch.cuda.synchronize()
        assert torch.equal(f.idx.long(), R.choose(l.double(), 4, "softmax"))
        assert bool((f.ws[f.need:] == 0xA5).all())
        f.ids = f.idx.long()
        _backward(f, None, 1.0, 1.0, check=False)
    torch.cuda.synchronize()


def test_workgroup_caps_change_nothing():
    s = torch.cuda.Stream()
    gen = _gen(14)
    l = _logits(1500, 256, "fp32", gen)
    dw = torch.randn(1500, 8, generator=gen, device=DEV)
    seq = torch.tensor([0, 100, 1400], dtype=torch.int32, device=DEV)
    want = Forward(l, 8, "softmax", seq=seq)().check()
    dwant = _backward(want, dw, 1.0, 0.5)
    try:
        for cap in (1, 3, 64):
            B.ep_set_workgroup_limit(s, cap)
            f = Forward(l, 8, "softmax", seq=seq)
            torch.cuda.synchronize()
            f(s).check()
            assert torch.equal(f.w, want.w) and torch.equal(f.losses, want.losses)
            assert torch.equal(_backward(f, dw, 1.0, 0.5, stream=s), dwant)
    finally:
        torch.cuda.synchronize()
        B.ep_set_workgroup_limit(s, 0)


def test_two_streams_at_once():
    gen = _gen(15)
    streams = [torch.cuda.Stream() for _ in range(2)]
    calls = [Forward(_logits(6000, 256, "fp32", gen), 8, "softmax"), Forward(_logits(5000, 100, "bf16", gen), 4, "sigmoid")]
    torch.cuda.synchronize()
    for _ in range(5):
        for f, s in zip(calls, streams):
            f(s)
    for f in calls:
        f.check()


def test_graph_replays_on_new_inputs():
    gen = _gen(16)
    T, E, K = 700, 256, 8
    l = _logits(T, E, "fp32", gen)
    seq = torch.tensor([0, 300, 700], dtype=torch.int32, device=DEV)
    f = Forward(l, K, "softmax", seq=seq)
    dw = torch.randn(T, K, generator=gen, device=DEV)
    d, one = torch.empty_like(l), torch.ones(1, device=DEV)

    def both(stream):
        f(stream)
        B.ep_router_backward(f.l, f.idx, f.seq, f.counts, f.tokens, dw, one, one, T, E, K, f.S, B.EP_FP32, B.EP_SOFTMAX, 1, 1.0, d, stream)

    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    both(s)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        both(torch.cuda.current_stream())
    for k in range(4):
        l.copy_(_logits(T, E, "fp32", gen))
        d.fill_(-7.0)
        graph.replay()
        f.check()
        want, err = R.backward(l.double(), f.ids, "softmax", True, 1.0, dw, seq, f.counts, f.tokens, 1.0, 1.0)
        R.near(d, want, err, torch.float32)


def test_the_same_call_gives_the_same_bits():
    l = _logits(30000, 256, "fp32", _gen(17))
    a, b = Forward(l, 8, "softmax")(), Forward(l, 8, "softmax")()
    torch.cuda.synchronize()
    assert torch.equal(a.w, b.w) and torch.equal(a.losses, b.losses) and torch.equal(a.counts, b.counts)


def test_logits_behind_4_gib():
    T, E, K = (1 << 21) + 900, 1024, 2
    _say(f"[large] {T} x {E} bf16")
    l = torch.empty(T, E, dtype=torch.bfloat16, device=DEV).normal_(0, 1.5, generator=_gen(18))
    f = Forward(l, K, "softmax")()
    d = torch.empty_like(l)
    dw = torch.randn(T, K, generator=_gen(19), device=DEV)
    one = torch.ones(1, device=DEV)
    B.ep_router_backward(l, f.idx, None, f.counts, f.tokens, dw, one, None, T, E, K, 1, B.EP_BF16, B.EP_SOFTMAX, 1, 1.0, d)
    torch.cuda.synchronize()
    for rows in (slice(0, 500), slice(T - 2000, T)):
        part = l[rows].double()
        ids = R.choose(part, K, "softmax")
        assert torch.equal(f.idx[rows].long(), ids)
        w, err = R.weights(part, ids, "softmax", True, 1.0)
        R.near(f.w[rows], w, err, torch.float32)
        n = ids.shape[0]
        # the whole batch's counts and tokens, as one sequence that these rows belong to
        want, err = R.backward(part, ids, "softmax", True, 1.0, dw[rows], torch.tensor([0, n]), f.counts, f.tokens, 1.0, None)
        R.near(d[rows], want, err, torch.bfloat16)
    assert int(f.tokens[0]) == T and int(f.counts.sum()) == T * K


def test_the_routers_ids_and_weights_through_the_layer():
    """ep_router -> ep_layout: counts and slots of the router's own ids, its counts the layout's."""
    T, E, K = 333, 64, 8
    gen = _gen(20)
    mask = (torch.rand(T, generator=gen, device=DEV) > 0.1).to(torch.uint8)
    f = Forward(_logits(T, E, "fp32", gen), K, "sigmoid", scale=2.5, mask=mask, bias=torch.randn(E, generator=gen, device=DEV) * 0.1)()
    counts, offsets, dst = _ints((E,)), _ints((E + 1,)), _ints((T, K))
    meta, n = _ints((T, K + 2)), _ints((1,))
    wsb = B.ep_layout_workspace_bytes(T, K, E)
    ws = torch.empty(max(wsb, 16), dtype=torch.uint8, device=DEV)
    B.ep_layout(f.idx, T, K, E, 1, T * K, counts, offsets, dst, meta, n, ws, wsb)
    f.check()
    assert torch.equal(counts, f.counts[0]) and int(n) == int(f.tokens[-1]) == int(mask.sum())
    assert torch.equal(dst >= 0, f.idx >= 0)
