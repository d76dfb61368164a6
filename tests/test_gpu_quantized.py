"""The 8-bit integer operators on the GPU against plain 64-bit forms.

Codes of ep_quantize_rows, and results of ep_quantized_matmul, are determined to the last bit and have
to be equal. Rows per expert sit around the kernels' tiles (0, 1, 16, 17, 32, 33, 64, 128, 129, 300),
widths end inside steps and tiles, padding rows hold garbage and must neither be read nor written, spans
leave the buffer at either end.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - only on CPU hosts
    pytest.skip("needs a GPU", allow_module_level=True)

from combine_ep_layout_amd import binding as B  # noqa: E402
from tests import experts_ref as X  # noqa: E402

DEV = "cuda:0"
KIND = {"bf16": B.EP_BF16, "fp32": B.EP_FP32}
TYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}
NAN, INF, LEAST = float("nan"), float("inf"), 2.0 ** -100


def _say(msg):
    print(msg, flush=True)


def _gen(*seed):
    n = 0
    for s in seed:
        n = n * 1000003 + int(s)
    return torch.Generator(device=DEV).manual_seed(n % (1 << 62))


def _codes(shape, gen):
    return torch.randint(-128, 128, shape, generator=gen, device=DEV, dtype=torch.int8)


def _spans(counts, A, extra=0):
    off = [0]
    for c in counts:
        off.append(off[-1] + -(-c // A) * A)
    cap = off[-1] + extra
    rows = [range(o, o + c) for o, c in zip(off, counts)]
    real = torch.zeros(cap, dtype=torch.bool, device=DEV)
    for r in rows:
        real[r.start:r.stop] = True
    return (torch.tensor(counts, dtype=torch.int32, device=DEV), torch.tensor(off, dtype=torch.int32, device=DEV), rows, real, cap)


# ------------------------------------------------------------------ ep_quantized_matmul

def _exact(x, sx, w, sw, out):
    """The result to the last bit: an exact sum, rounded to binary32, scaled twice, rounded to the type."""
    total = x.double() @ w.double().T  # below 2^53: exact
    return (total.float() * sx[:, None] * sw).to(out)


def _matmul(x, sx, w, sw, c, o, E, cap, y, stream=None):
    N, K = w.shape[1:]
    B.ep_quantized_matmul(x, sx, sx.shape[1], w, sw, c, o, E, cap, K, N, y, KIND["fp32" if y.dtype == torch.float32 else "bf16"], stream)


MATMUL = [
    # K, N, counts, A, y type, scale columns
    (16, 8, [1], 1, "fp32", 1),
    (64, 24, [3, 0, 17], 4, "bf16", 1),
    (80, 40, [1, 2, 1], 1, "fp32", 3),
    (208, 520, [0, 1, 15, 16, 33, 65, 0], 8, "bf16", 1),
    (7168, 72, [2, 5], 1, "fp32", 56),
    (1024, 1048, [16, 31, 130, 0, 1], 16, "fp32", 1),
    (2064, 264, [300, 0, 129], 128, "bf16", 1),
    (512, 4096, [1, 40, 0, 0, 3], 16, "bf16", 2),
    (144, 136, [1, 0, 16, 17, 32, 33, 70, 2, 64, 63, 96, 127, 128, 255, 256, 257] * 2, 1, "fp32", 1),
    (320, 776, [100] * 9, 1, "bf16", 1),
    (4096, 512, [700], 1, "bf16", 1),
    (96, 2056, [513, 1, 255], 1, "fp32", 1),
    (7168, 4096, [1], 1, "bf16", 1),
    (2048, 1032, [0, 0, 900, 0], 128, "fp32", 1),
    (128, 16, [5000], 1, "bf16", 1),
]


@pytest.mark.parametrize("K,N,counts,A,out,cols", MATMUL)
def test_matmul(K, N, counts, A, out, cols):
    _say(f"[matmul] K={K} N={N} counts={counts} A={A} {out} cols={cols}")
    gen = _gen(1, K, N, len(counts))
    E = len(counts)
    c, o, rows, real, cap = _spans(counts, A, 5)
    x, w = _codes((cap, K), gen), _codes((E, N, K), gen)
    sx = torch.rand(cap, cols, generator=gen, device=DEV) + 0.1
    sx[~real] = NAN
    sw = torch.randn(E, N, generator=gen, device=DEV)
    y = torch.full((cap, N), -7.0, dtype=TYPE[out], device=DEV)
    _matmul(x, sx, w, sw, c, o, E, cap, y)
    torch.cuda.synchronize()
    for e, r in enumerate(rows):
        if len(r):
            s = slice(r.start, r.stop)
            assert torch.equal(y[s], _exact(x[s], sx[s, 0], w[e], sw[e], TYPE[out])), f"expert {e}"
    assert bool((y[~real] == -7.0).all()), "rows behind an expert's last are left alone"


@pytest.mark.parametrize("rows,K,N", [(1, 7168, 4096), (5, 512, 200), (200, 1040, 264), (1, 16, 8), (1000, 2048, 1024)])
def test_matmul_of_one_matrix_without_routing_arrays(rows, K, N):
    _say(f"[matmul dense] rows={rows} K={K} N={N}")
    gen = _gen(2, K, N, rows)
    x, w = _codes((rows, K), gen), _codes((1, N, K), gen)
    sx, sw = torch.rand(rows, 1, generator=gen, device=DEV), torch.rand(1, N, generator=gen, device=DEV)
    y = torch.empty(rows, N, device=DEV)
    _matmul(x, sx, w, sw, None, None, 1, rows, y)
    torch.cuda.synchronize()
    assert torch.equal(y, _exact(x, sx[:, 0], w[0], sw[0], torch.float32))


def test_matmul_of_the_largest_sums():
    """Every code -128 at the widest rows: 2^14 times the width, just below 2^31."""
    K = B.EP_MAX_QUANTIZED_WIDTH
    for rows in (2, 70, 300):
        x = torch.full((rows, K), -128, dtype=torch.int8, device=DEV)
        w = torch.full((1, 24, K), -128, dtype=torch.int8, device=DEV)
        w[0, 1] = 127
        y = torch.empty(rows, 24, device=DEV)
        one = torch.ones(rows, 1, device=DEV)
        _matmul(x, one, w, torch.ones(1, 24, device=DEV), None, None, 1, rows, y)
        torch.cuda.synchronize()
        want = torch.full((24,), 16384.0 * K, device=DEV)
        want[1] = float(torch.tensor(-128.0 * 127 * K))
        assert torch.equal(y, want.expand(rows, 24))


def test_matmul_of_scales_that_are_no_numbers():
    x, w = _codes((40, 64), _gen(3)), _codes((1, 64, 64), _gen(4))
    sx = torch.ones(40, 1, device=DEV)
    sx[3], sx[4], sx[5] = NAN, INF, 0.0
    y = torch.empty(40, 64, device=DEV)
    _matmul(x, sx, w, torch.ones(1, 64, device=DEV), None, None, 1, 40, y)
    torch.cuda.synchronize()
    want = _exact(x, sx[:, 0], w[0], torch.ones(64, device=DEV), torch.float32)
    assert torch.equal(torch.nan_to_num(y, 1.5), torch.nan_to_num(want, 1.5))
    assert bool(torch.isnan(y[3]).all()) and not bool(torch.isnan(y[6:]).any())


SPANS = [([4, 9, 5, 3, -2], [0, 16, 40, -3, 8, 10]), ([50, 200, 2 ** 31 - 1], [-20, 10, 30, 40]), ([300], [-100, 0]), ([7, 0], [2 ** 31 - 1, 0, 0])]


@pytest.mark.parametrize("counts,offsets", SPANS)
def test_matmul_spans_that_leave_the_buffer_are_cut(counts, offsets):
    _say(f"[matmul spans] {counts} {offsets}")
    gen = _gen(5)
    K, N, cap, E = 256, 72, 120, len(counts)
    room = 40  # rows around the buffer, which hold a sentinel
    x, w = _codes((cap, K), gen), _codes((E, N, K), gen)
    sx, sw = torch.rand(cap, 1, generator=gen, device=DEV), torch.rand(E, N, generator=gen, device=DEV)
    whole = torch.full((cap + 2 * room, N), -7.0, device=DEV)
    y = whole[room:room + cap]
    c, o = (torch.tensor(v, dtype=torch.int32, device=DEV) for v in (counts, offsets))
    _matmul(x, sx, w, sw, c, o, E, cap, y)
    torch.cuda.synchronize()
    left = torch.ones(cap, dtype=torch.bool, device=DEV)
    for e in range(E):
        b, n = max(offsets[e], 0), min(offsets[e] + counts[e], cap)
        if b < n:
            left[b:n] = False
    last = {}
    for e in range(E):  # where spans overlap, either is right: check rows of one span
        for r in range(max(offsets[e], 0), min(offsets[e] + counts[e], cap)):
            last.setdefault(r, []).append(e)
    for r, es in last.items():
        if len(es) == 1:
            assert torch.equal(y[r], _exact(x[r:r + 1], sx[r:r + 1, 0], w[es[0]], sw[es[0]], torch.float32)[0]), (r, es)
    assert bool((y[left] == -7.0).all()) and bool((whole[:room] == -7.0).all()) and bool((whole[room + cap:] == -7.0).all())


def test_matmul_1024_experts():
    gen = _gen(6)
    E, K, N = 1024, 128, 40
    counts = torch.randint(0, 4, (E,), generator=gen, device=DEV).tolist()
    counts[3], counts[900] = 140, 77
    c, o, rows, real, cap = _spans(counts, 4)
    x, w = _codes((cap, K), gen), _codes((E, N, K), gen)
    sx, sw = torch.rand(cap, 1, generator=gen, device=DEV), torch.rand(E, N, generator=gen, device=DEV)
    y = torch.full((cap, N), -7.0, device=DEV)
    _matmul(x, sx, w, sw, c, o, E, cap, y)
    torch.cuda.synchronize()
    expert = torch.searchsorted(o[1:].long(), torch.arange(cap, device=DEV), right=True).clamp(max=E - 1)
    total = torch.zeros(cap, N, dtype=torch.float64, device=DEV)
    for b in range(0, cap, 256):
        s = slice(b, b + 256)
        total[s] = (w[expert[s]].double() * x[s].double()[:, None]).sum(2)
    want = total.float() * sx * sw[expert]
    assert torch.equal(y[real], want[real]) and bool((y[~real] == -7.0).all())


def test_matmul_behind_4_gib():
    gen = _gen(7)
    K, N = 1024, 64
    rows = (1 << 22) + 500  # x just over 4 GiB
    _say(f"[matmul large] rows={rows}")
    x = torch.empty(rows, K, dtype=torch.int8, device=DEV)
    x[:1000], x[-1000:] = _codes((1000, K), gen), _codes((1000, K), gen)
    counts, offsets = [600, 0, 700], [0, 600, rows - 700, rows]
    w = _codes((3, N, K), gen)
    sx, sw = torch.rand(rows, 1, generator=gen, device=DEV), torch.rand(3, N, generator=gen, device=DEV)
    y = torch.full((rows, N), -7.0, dtype=torch.bfloat16, device=DEV)
    c, o = (torch.tensor(v, dtype=torch.int32, device=DEV) for v in (counts, offsets))
    _matmul(x, sx, w, sw, c, o, 3, rows, y)
    torch.cuda.synchronize()
    assert torch.equal(y[:600], _exact(x[:600], sx[:600, 0], w[0], sw[0], torch.bfloat16))
    assert torch.equal(y[-700:], _exact(x[-700:], sx[-700:, 0], w[2], sw[2], torch.bfloat16))
    assert bool((y[600:-700] == -7.0).all())


def test_matmul_weights_behind_4_gib():
    E, K, N = 5, 16384, 65536  # 1 GiB each
    gen = _gen(8)
    w = torch.zeros(E, N, K, dtype=torch.int8, device=DEV)
    w[4, -200:] = _codes((200, K), gen)
    x = _codes((3, K), gen)
    c, o = torch.tensor([0, 0, 0, 0, 3], dtype=torch.int32, device=DEV), torch.tensor([0, 0, 0, 0, 0, 3], dtype=torch.int32, device=DEV)
    sx, sw = torch.rand(3, 1, generator=gen, device=DEV), torch.rand(E, N, generator=gen, device=DEV)
    y = torch.full((3, N), -7.0, device=DEV)
    _matmul(x, sx, w, sw, c, o, E, 3, y)
    torch.cuda.synchronize()
    assert torch.equal(y[:, -200:], _exact(x, sx[:, 0], w[4, -200:], sw[4, -200:], torch.float32)) and bool((y[:, :-200] == 0).all())


def test_matmul_caps_streams_and_graph_replays():
    gen = _gen(9)
    counts = [0, 1, 33, 300, 17, 64]
    c, o, rows, real, cap = _spans(counts, 8)
    E, K, N = len(counts), 528, 776
    x, w = _codes((cap, K), gen), _codes((E, N, K), gen)
    sx, sw = torch.rand(cap, 1, generator=gen, device=DEV), torch.rand(E, N, generator=gen, device=DEV)
    want = torch.full((cap, N), -7.0, device=DEV)
    _matmul(x, sx, w, sw, c, o, E, cap, want)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    try:
        for cap_ in (1, 3, 64):
            _say(f"[matmul cap] {cap_}")
            B.ep_set_workgroup_limit(s, cap_)
            y = torch.full((cap, N), -7.0, device=DEV)
            torch.cuda.synchronize()
            _matmul(x, sx, w, sw, c, o, E, cap, y, s)
            s.synchronize()
            assert torch.equal(y, want)
    finally:
        torch.cuda.synchronize()
        B.ep_set_workgroup_limit(s, 0)
    y = torch.empty(cap, N, device=DEV)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        _matmul(x, sx, w, sw, c, o, E, cap, y, torch.cuda.current_stream())
    for k in range(3):  # new rows and new routing
        x.copy_(_codes((cap, K), gen))
        n = [5 * k, 100, 0, 7 + k, 0, 130]
        c2, o2, rows2, real2, _ = _spans(n, 8)
        c.copy_(c2)
        o.copy_(o2)
        y.fill_(-7.0)
        graph.replay()
        torch.cuda.synchronize()
        for e, r in enumerate(rows2):
            q = slice(r.start, r.stop)
            assert torch.equal(y[q], _exact(x[q], sx[q, 0], w[e], sw[e], torch.float32))
        assert bool((y[:real2.numel()][~real2] == -7.0).all()) and bool((y[real2.numel():] == -7.0).all())


# ------------------------------------------------------------------ ep_quantize_rows, ep_swiglu_quantize

def _quantized(v):
    """(codes, scales) of rows of binary32 values by the definition: the factor in binary32, its product exact."""
    bad = ~torch.isfinite(v).all(1)
    top = torch.where(bad, 0.0, torch.nan_to_num(v.abs()).amax(1)).clamp(min=LEAST)
    # quotients of binary32 numbers rounded to 64 and then to 32 bits are rounded as if once
    by, scale = (torch.full_like(top, 127.0).double() / top.double()).float(), (top.double() / 127.0).float()
    code = torch.round(torch.where(bad[:, None], 0.0, v.double()) * by.double()[:, None])
    return code.to(torch.int8), torch.where(bad, NAN, scale)


def _same(a, b):
    return torch.equal(torch.nan_to_num(a, -3.0), torch.nan_to_num(b, -3.0))


WIDTHS = [16, 48, 128, 272, 512, 1008, 1024, 1040, 1408, 2048, 2064, 4096, 7168, 8192, 8208, 20000, 40000]


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("W", WIDTHS)
def test_quantize_rows(W, kind):
    _say(f"[quantize] W={W} {kind}")
    gen = _gen(10, W)
    counts = [0, 1, 5, 33, 0, 70, 2]
    c, o, rows, real, cap = _spans(counts, 8, 3)
    x = (torch.randn(cap, W, generator=gen, device=DEV) * torch.exp2(torch.randint(-90, 90, (cap, 1), generator=gen, device=DEV).float())).to(TYPE[kind])
    x[0] = 0.0
    x[8, 3] = INF
    x[9, W - 1] = NAN
    x[10] = 1e-38
    x[11] = torch.finfo(TYPE[kind]).max
    x[12, :] = 0.5
    x[12, 0] = -1.0            # halves of the largest: 63.5 steps
    x[13] = (torch.arange(W, device=DEV) % 255 - 127).to(TYPE[kind])
    x[13, 0] = 127.0
    x[~real] = NAN
    for cols in (1, 5):
        codes = torch.full((cap, W), 99, dtype=torch.int8, device=DEV)
        scales = torch.full((cap, cols), -7.0, device=DEV)
        B.ep_quantize_rows(x, c, o, len(counts), cap, W, KIND[kind], codes, scales, cols)
        torch.cuda.synchronize()
        want, scale = _quantized(x.float())
        assert torch.equal(codes[real], want[real]), f"rows {torch.nonzero((codes != want).any(1) & real)[:4].flatten().tolist()}"
        assert _same(scales[real], scale[real][:, None].expand(-1, cols))
        assert bool((codes[~real] == 99).all()) and bool((scales[~real] == -7.0).all())


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("W", WIDTHS[:-2])
def test_swiglu_quantize(W, kind):
    _say(f"[swiglu quantize] W={W} {kind}")
    gen = _gen(11, W)
    counts = [0, 1, 5, 33, 0, 30, 2]
    c, o, rows, real, cap = _spans(counts, 8, 3)
    v = (torch.randn(cap, 2 * W, generator=gen, device=DEV) * 2).to(TYPE[kind])
    v[8, 3] = INF
    v[9, 2 * W - 1] = NAN
    v[10, :W] = -95.0
    v[10, W:] = 1e30
    v[11] = 0.0
    v[12, :W] *= 20
    v[~real] = NAN
    codes = torch.full((cap, W), 99, dtype=torch.int8, device=DEV)
    scales = torch.full((cap, 2), -7.0, device=DEV)
    B.ep_swiglu_quantize(v, c, o, len(counts), cap, W, KIND[kind], codes, scales, 2)
    torch.cuda.synchronize()
    assert bool((codes[~real] == 99).all()) and bool((scales[~real] == -7.0).all())
    assert bool(torch.isnan(scales[[8, 9]]).all()) and bool((codes[[8, 9]] == 0).all())
    real[8] = real[9] = False
    g, u = v[real].double().split(W, 1)
    zero = torch.zeros_like(g)
    h, dh = X.gated(g, zero, u, zero)
    top, dtop = h.abs().amax(1).clamp(min=LEAST), dh.amax(1)
    # the scale: the largest within its error, and the division's rounding
    for col in (0, 1):
        assert bool(((scales[real][:, col].double() - top / 127).abs() <= (dtop + 2 * X.U * top) / 127).all())
    # a code: within half a step of h over the scale; 127 / a and its product's bounds as above, all over the scale
    at = h * (127 / top)[:, None]
    slack = dh * (127 / top)[:, None] + at.abs() * ((dtop / top)[:, None] + 4 * X.U)
    assert bool(((codes[real].double() - at).abs() <= 0.5 + slack).all())
    assert int(codes[real].double().abs().amax()) <= 127


@pytest.mark.parametrize("fn,factor", [(B.ep_quantize_rows, 1), (B.ep_swiglu_quantize, 2)], ids=["rows", "gated"])
def test_quantize_without_routing_arrays_caps_and_replays(fn, factor):
    gen = _gen(12)
    R, W = 500, 1040
    x = torch.randn(R, factor * W, generator=gen, device=DEV).bfloat16()
    want = [torch.empty(R, W, dtype=torch.int8, device=DEV), torch.empty(R, 1, device=DEV)]
    fn(x, None, None, 1, R, W, B.EP_BF16, *want, 1)
    torch.cuda.synchronize()
    if factor == 1:
        codes, scales = _quantized(x.float())
        assert torch.equal(want[0], codes) and torch.equal(want[1][:, 0], scales)
    s = torch.cuda.Stream()
    got = [torch.empty_like(t) for t in want]
    try:
        for cap in (1, 7):
            B.ep_set_workgroup_limit(s, cap)
            for t in got:
                t.zero_()
            torch.cuda.synchronize()
            fn(x, None, None, 1, R, W, B.EP_BF16, *got, 1, s)
            s.synchronize()
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    finally:
        torch.cuda.synchronize()
        B.ep_set_workgroup_limit(s, 0)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        fn(x, None, None, 1, R, W, B.EP_BF16, *got, 1, torch.cuda.current_stream())
    for _ in range(3):
        x.copy_(torch.randn(R, factor * W, generator=gen, device=DEV).bfloat16())
        fn(x, None, None, 1, R, W, B.EP_BF16, *want, 1)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("counts,offsets", SPANS)
def test_quantize_spans_that_leave_the_buffer_are_cut(counts, offsets):
    gen = _gen(13)
    cap, W, room, E = 120, 64, 40, len(counts)
    x = torch.randn(cap, W, generator=gen, device=DEV)
    whole = torch.full((cap + 2 * room, W), 99, dtype=torch.int8, device=DEV)
    scales = torch.full((cap + 2 * room, 1), -7.0, device=DEV)
    c, o = (torch.tensor(v, dtype=torch.int32, device=DEV) for v in (counts, offsets))
    B.ep_quantize_rows(x, c, o, E, cap, W, B.EP_FP32, whole[room:room + cap], scales[room:room + cap], 1)
    torch.cuda.synchronize()
    real = torch.zeros(cap + 2 * room, dtype=torch.bool, device=DEV)
    for b, n in zip(offsets, counts):
        real[room + min(max(b, 0), cap):room + max(min(b + n, cap), 0)] = True
    want, scale = _quantized(x)
    assert torch.equal(whole[real], want[real[room:room + cap]]) and torch.equal(scales[real][:, 0], scale[real[room:room + cap]])
    assert bool((whole[~real] == 99).all()) and bool((scales[~real] == -7.0).all())


@pytest.mark.parametrize("E,W,kind,rows", [(1024, 32, "fp32", 90000), (300, 2064, "bf16", 14000), (70, 20000, "bf16", 3500), (256, 512, "bf16", 40000)])
def test_quantize_many_ragged_experts(E, W, kind, rows):
    """More rows than workgroups take at once, experts in no order, some of them without rows, padding between."""
    _say(f"[quantize many] E={E} W={W} {kind} rows={rows}")
    gen = _gen(14, E, W)
    share = torch.rand(E, generator=gen, device=DEV) ** 3
    share[torch.rand(E, generator=gen, device=DEV) < 0.3] = 0
    counts = (share / share.sum() * rows).to(torch.int32)
    order = torch.randperm(E, generator=gen, device=DEV)
    room = (counts[order] + 40 + 7) // 8 * 8
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[order] = (torch.cumsum(room, 0) - room).to(torch.int32)
    cap = int(room.sum())
    real = torch.zeros(cap, dtype=torch.bool, device=DEV)
    for b, n in zip(offsets.tolist(), counts.tolist()):
        real[b:b + n] = True
    x = torch.randn(cap, W, generator=gen, device=DEV).to(TYPE[kind])
    x[~real] = NAN
    want, scale = _quantized(x[real].float())
    for limit in (0, 3):
        codes = torch.full((cap, W), 99, dtype=torch.int8, device=DEV)
        scales = torch.full((cap, 1), -7.0, device=DEV)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        if limit:
            B.ep_set_workgroup_limit(s, limit)
        B.ep_quantize_rows(x, counts, offsets, E, cap, W, KIND[kind], codes, scales, 1, s)
        s.synchronize()
        if limit:
            B.ep_set_workgroup_limit(s, 0)
        assert torch.equal(codes[real], want) and torch.equal(scales[real][:, 0], scale)
        assert bool((codes[~real] == 99).all()) and bool((scales[~real] == -7.0).all())


def test_quantize_behind_4_gib():
    R, W = (1 << 20) + 70, 4096  # codes just over 4 GiB
    _say(f"[quantize large] {R} x {W}")
    x = torch.empty(R, W, dtype=torch.bfloat16, device=DEV)
    x.normal_(0, 1, generator=_gen(14))
    codes = torch.empty(R, W, dtype=torch.int8, device=DEV)
    scales = torch.empty(R, 1, device=DEV)
    B.ep_quantize_rows(x, None, None, 1, R, W, B.EP_BF16, codes, scales, 1)
    torch.cuda.synchronize()
    for s in (slice(0, 100), slice(R - 500, R)):
        want, scale = _quantized(x[s].float())
        assert torch.equal(codes[s], want) and torch.equal(scales[s, 0], scale)


# ------------------------------------------------------------------ the whole layer

@pytest.mark.parametrize("T,E,K,A,H,I", [(1, 16, 4, 1, 512, 256), (100, 16, 4, 16, 1024, 272), (700, 8, 2, 128, 512, 640)])
def test_the_layer_in_8_bit_integers(T, E, K, A, H, I):
    """ep_router, ep_quantize_rows, ep_layout_dispatch (codes and scale rows), ep_quantized_matmul, ep_swiglu_quantize,
    ep_quantized_matmul, ep_combine as they would be used; each stage against 64 bits on what it was given."""
    _say(f"[int8 layer] T={T} E={E} K={K} A={A} H={H} I={I}")
    gen = _gen(15, T, H, I)
    cap, S = T * K + E * (A - 1), H // 128
    x = torch.randn(T, H, generator=gen, device=DEV).bfloat16()
    logits = torch.randn(T, E, generator=gen, device=DEV)
    w_in, w_out = torch.randn(E, 2 * I, H, generator=gen, device=DEV) * H ** -0.5, torch.randn(E, H, I, generator=gen, device=DEV) * I ** -0.5
    q = {}
    for name, w in (("in", w_in), ("out", w_out)):  # a weight matrix is quantised by rows: one scale per channel
        q[name] = torch.empty(w.shape, dtype=torch.int8, device=DEV), torch.empty(w.shape[:2], device=DEV)
        B.ep_quantize_rows(w, None, None, 1, w.shape[0] * w.shape[1], w.shape[2], B.EP_FP32, *q[name], 1)
    idx, wts = torch.empty(T, K, dtype=torch.int32, device=DEV), torch.empty(T, K, device=DEV)
    B.ep_router(logits, None, None, None, T, E, K, 1, B.EP_FP32, B.EP_SOFTMAX, 1, 1.0, 0, idx, wts)
    codes, scales = torch.empty(T, H, dtype=torch.int8, device=DEV), torch.empty(T, S, device=DEV)
    B.ep_quantize_rows(x, None, None, 1, T, H, B.EP_BF16, codes, scales, S)
    counts, offsets, dst = (torch.empty(n, dtype=torch.int32, device=DEV) for n in ((E,), (E + 1,), (T, K)))
    meta, nrecv = torch.empty(T, K + 2, dtype=torch.int32, device=DEV), torch.empty(1, dtype=torch.int32, device=DEV)
    wsb = B.ep_layout_dispatch_workspace_bytes(T, K, E)
    ws = torch.empty(max(wsb, 16), dtype=torch.uint8, device=DEV)
    ex, es = torch.full((cap, H), 55, dtype=torch.int8, device=DEV), torch.full((cap, S), NAN, device=DEV)
    B.ep_layout_dispatch(idx, T, K, E, A, cap, counts, offsets, dst, meta, nrecv, ws, wsb, codes, scales, None, H, B.EP_FP8_E4M3, ex, es, None)
    z = torch.zeros(cap, 2 * I, dtype=torch.bfloat16, device=DEV)
    B.ep_quantized_matmul(ex, es, S, *q["in"], counts, offsets, E, cap, H, 2 * I, z, B.EP_BF16)
    h, hs = torch.zeros(cap, I, dtype=torch.int8, device=DEV), torch.zeros(cap, 1, device=DEV)
    B.ep_swiglu_quantize(z, counts, offsets, E, cap, I, B.EP_BF16, h, hs, 1)
    y = torch.zeros(cap, H, dtype=torch.bfloat16, device=DEV)
    B.ep_quantized_matmul(h, hs, 1, *q["out"], counts, offsets, E, cap, I, H, y, B.EP_BF16)
    out = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    B.ep_combine(y, wts, None, dst, T, H, K, B.EP_BF16, cap, out)
    torch.cuda.synchronize()

    want, scale = _quantized(x.float())
    assert torch.equal(codes, want) and torch.equal(scales, scale[:, None].expand(-1, S))
    flat, slot = idx.long().flatten(), dst.long().flatten()
    token = torch.arange(T, device=DEV).repeat_interleave(K)
    for e in range(E):
        r = slot[flat == e]
        if not r.numel():
            continue
        assert torch.equal(ex[r], codes[token[flat == e]])
        assert torch.equal(z[r], _exact(ex[r], es[r, 0], q["in"][0][e], q["in"][1][e], torch.bfloat16))
        g, u = z[r].double().split(I, 1)
        act = g * torch.sigmoid(g) * u
        assert bool(((h[r].double() * hs[r].double() - act).abs() <= hs[r].double() * 0.51).all())  # half a step; 0.01 of one for the activation
        assert torch.equal(y[r], _exact(h[r], hs[r, 0], q["out"][0][e], q["out"][1][e], torch.bfloat16))
    p = (y[slot].double() * wts.flatten().double()[:, None]).view(T, K, H)
    bound = (K + 2) * X.U * p.abs().sum(1) + 2.0 ** -8 * p.sum(1).abs() * 1.01
    assert bool(((out.double() - p.sum(1)).abs() <= bound).all())
    # and the layer as a whole stands for the layer of its unquantised weights: a step of 1/127 of a row's
    # largest in x, w_in, h and w_out each; statistically a few percent, so this only finds what is plainly wrong
    exact = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    for e in range(E):
        t, k = torch.nonzero(idx == e, as_tuple=True)
        g, u = (x[t].double() @ w_in[e].double().T).split(I, 1)
        exact.index_add_(0, t, (g * torch.sigmoid(g) * u) @ w_out[e].double().T * wts[t, k].double()[:, None])
    assert float((out.double() - exact).norm() / exact.norm()) < 0.1
