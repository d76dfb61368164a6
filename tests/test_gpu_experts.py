"""The experts' operators on the GPU against plain 64-bit forms.

Shapes sit where the kernels can go wrong: rows per expert around the 16-row
tiles (0, 1, 15, 16, 17, 33, 65), widths that end inside a step of 128, output
columns that end inside a tile, padding rows (which hold NaN on entry and must
neither be read nor written), spans that leave the buffer, masked and repeated
ids, workgroup caps, other streams and graph replays.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - only on CPU hosts
    pytest.skip("needs a GPU", allow_module_level=True)

from combine_ep_layout_amd import binding as B  # noqa: E402
from tests import experts_ref as R  # noqa: E402

DEV = "cuda:0"
KIND = {"bf16": B.EP_BF16, "fp32": B.EP_FP32, "fp8": B.EP_FP8_E4M3, "fp4": B.EP_FP4X2}
TYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}
NAN = float("nan")


def _say(msg):
    print(msg, flush=True)


def _gen(*seed):
    n = 0
    for s in seed:
        n = n * 1000003 + int(s)
    return torch.Generator(device=DEV).manual_seed(n % (1 << 62))


def _normal(shape, gen, std=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=gen, device=DEV) * std).to(dtype)


def _weights(E, N, K, kind, gen):
    """(weights, scales): scales that are no powers of two and differ from row to row."""
    if kind == "bf16":
        return _normal((E, N, K), gen, K ** -0.5, torch.bfloat16), None
    scales = (torch.rand(E, N, K // 128, generator=gen, device=DEV) + 0.3) * K ** -0.5
    if kind == "fp8":
        return _normal((E, N, K), gen, 2.0).to(torch.float8_e4m3fn).view(torch.uint8), scales
    return torch.randint(0, 256, (E, N, K // 2), generator=gen, device=DEV, dtype=torch.uint8), scales


def _spans(counts, A, cap=None):
    """counts and offsets on the device, the real rows of every expert, and the capacity."""
    off = [0]
    for c in counts:
        off.append(off[-1] + -(-c // A) * A)
    cap = off[-1] if cap is None else cap
    rows = [range(min(o, cap), min(o + c, cap)) for o, c in zip(off, counts)]
    return (torch.tensor(counts, dtype=torch.int32, device=DEV),
            torch.tensor(off, dtype=torch.int32, device=DEV), rows, cap)


def _real(rows, cap):
    live = torch.zeros(cap, dtype=torch.bool, device=DEV)
    for r in rows:
        live[r.start:r.stop] = True
    return live


# ------------------------------------------------------------------ ep_expert_matvec

MATVEC = [
    # kind, K, N, counts, A, y type
    ("bf16", 8, 8, [1], 1, "bf16"),
    ("bf16", 136, 24, [3, 0, 17], 4, "fp32"),
    ("bf16", 1160, 520, [0, 1, 15, 16, 33, 65, 0], 8, "bf16"),
    ("bf16", 7168, 72, [2, 5], 1, "fp32"),
    ("fp8", 128, 40, [1, 0, 2], 1, "bf16"),
    ("fp8", 896, 1048, [16, 31, 130, 0, 1], 16, "fp32"),
    ("fp4", 128, 8, [1], 1, "fp32"),
    ("fp4", 384, 88, [17, 0, 4, 64, 65], 1, "fp32"),
    ("fp4", 2048, 4096, [1, 40, 0, 0, 3], 16, "bf16"),
]


# Enough tiles for the kernels that take 128 rows of a matrix at once: 40 experts x 8 tiles.
WIDE_COUNTS = [1, 0, 16, 17, 32, 33, 70, 2] * 5
MATVEC += [
    ("bf16", 1160, 904, WIDE_COUNTS, 8, "fp32"),
    ("bf16", 128, 1024, WIDE_COUNTS, 1, "bf16"),
    ("bf16", 24, 1000, WIDE_COUNTS, 1, "fp32"),
    ("fp8", 128, 904, WIDE_COUNTS, 1, "fp32"),
    ("fp8", 640, 912, WIDE_COUNTS, 16, "bf16"),
    ("fp4", 128, 904, WIDE_COUNTS, 1, "fp32"),
    ("fp4", 640, 904, WIDE_COUNTS, 4, "fp32"),
    ("fp4", 1024, 2056, WIDE_COUNTS, 1, "bf16"),
    ("bf16", 512, 1024, [100] * 9, 1, "bf16"),  # 72 tiles, many rows each
]


@pytest.mark.parametrize("kind,K,N,counts,A,out", MATVEC)
def test_matvec(kind, K, N, counts, A, out):
    _say(f"[matvec] {kind} K={K} N={N} counts={counts} A={A} {out}")
    gen = _gen(1, K, N, len(counts))
    E = len(counts)
    c, o, rows, cap = _spans(counts, A)
    w, s = _weights(E, N, K, kind, gen)
    x = torch.full((cap, K), NAN, dtype=torch.bfloat16, device=DEV)
    for r in rows:
        x[r.start:r.stop] = _normal((len(r), K), gen, 1.0, torch.bfloat16)
    y = torch.full((cap, N), -7.0, dtype=TYPE[out], device=DEV)
    B.ep_expert_matvec(x, w, s, c, o, E, cap, K, N, KIND[kind], y, KIND[out])
    torch.cuda.synchronize()
    for e, r in enumerate(rows):
        if len(r):
            xe = x[r.start:r.stop].double()
            want, err = R.product(xe, torch.zeros_like(xe), R.values(w[e], None if s is None else s[e], kind))
            R.near(y[r.start:r.stop], want, err, TYPE[out])
    assert bool((y[~_real(rows, cap)] == -7.0).all()), "rows behind an expert's last are left alone"


@pytest.mark.parametrize("kind,rows,K,N", [("fp4", 1, 7168, 4096), ("bf16", 1, 1024, 512), ("fp8", 5, 512, 200)])
def test_matvec_one_matrix_without_routing_arrays(kind, rows, K, N):
    _say(f"[matvec dense] {kind} rows={rows} K={K} N={N}")
    gen = _gen(2, K, N, rows)
    w, s = _weights(1, N, K, kind, gen)
    x = _normal((rows, K), gen, 1.0, torch.bfloat16)
    y = torch.empty(rows, N, device=DEV)
    B.ep_expert_matvec(x, w, s, None, None, 1, rows, K, N, KIND[kind], y, B.EP_FP32)
    torch.cuda.synchronize()
    want, err = R.product(x.double(), torch.zeros(rows, K, dtype=torch.float64, device=DEV),
                          R.values(w[0], None if s is None else s[0], kind))
    R.near(y, want, err, torch.float32)


def test_matvec_spans_that_leave_the_buffer_are_cut():
    """Offsets and counts beyond capacity_rows, and a negative offset, reach no memory outside."""
    gen = _gen(3)
    K, N, cap = 256, 64, 20
    c = torch.tensor([4, 9, 5, 3, -2], dtype=torch.int32, device=DEV)
    o = torch.tensor([0, 16, 40, -3, 8, 10], dtype=torch.int32, device=DEV)  # 16..25 is cut at 20
    w, s = _weights(5, N, K, "fp8", gen)
    x = _normal((cap, K), gen, 1.0, torch.bfloat16)
    y = torch.full((cap, N), -7.0, device=DEV)
    B.ep_expert_matvec(x, w, s, c, o, 5, cap, K, N, B.EP_FP8_E4M3, y, B.EP_FP32)
    torch.cuda.synchronize()
    for e, r in ((0, slice(0, 4)), (1, slice(16, 20))):
        want, err = R.product(x[r].double(), torch.zeros(4, K, dtype=torch.float64, device=DEV),
                              R.values(w[e], s[e], "fp8"))
        R.near(y[r], want, err, torch.float32)
    assert bool((y[4:16] == -7.0).all())


def test_matvec_many_experts_few_active():
    gen = _gen(4)
    E, K, N = 1024, 128, 48
    counts = [0] * E
    for e in (0, 3, 255, 256, 700, 1023):
        counts[e] = 1 + e % 3
    c, o, rows, cap = _spans(counts, 2)
    w, s = _weights(E, N, K, "bf16", gen)
    x = _normal((cap, K), gen, 1.0, torch.bfloat16)
    y = torch.full((cap, N), -7.0, device=DEV)
    B.ep_expert_matvec(x, w, s, c, o, E, cap, K, N, B.EP_BF16, y, B.EP_FP32)
    torch.cuda.synchronize()
    for e, r in enumerate(rows):
        if len(r):
            xe = x[r.start:r.stop].double()
            want, err = R.product(xe, torch.zeros_like(xe), w[e].double())
            R.near(y[r.start:r.stop], want, err, torch.float32)
    assert bool((y[~_real(rows, cap)] == -7.0).all())


# ---------------------------------------------------------------------- ep_moe_layer

def _route(T, K, E, masked, repeat, gen):
    idx = torch.rand(T, max(E, K), generator=gen, device=DEV).argsort(1)[:, :K] % E
    if repeat:
        idx[:, -1] = idx[:, 0]
    idx = idx.to(torch.int32)
    drop = torch.rand(T, K, generator=gen, device=DEV)
    idx[drop < masked] = -1
    idx[(drop >= masked) & (drop < masked * 1.2)] = E + 3  # also outside
    return idx.contiguous()


def _layer_case(T, K, E, H, I, kind, masked=0.0, repeat=False, seed=0):
    gen = _gen(5, T, K, E, H, I, seed)
    a = {"idx": _route(T, K, E, masked, repeat, gen), "x": _normal((T, H), gen, 1.0, torch.bfloat16),
         "probs": torch.softmax(_normal((T, K), gen), 1), "bias": _normal((T, H), gen, 0.5, torch.bfloat16)}
    a["w_in"], a["s_in"] = _weights(E, 2 * I, H, kind, gen)
    a["w_out"], a["s_out"] = _weights(E, H, I, kind, gen)
    a["out"] = torch.full((T, H), NAN, dtype=torch.bfloat16, device=DEV)
    a["ws"] = torch.full((B.ep_moe_layer_workspace_bytes(T, K, I),), 0xA5, dtype=torch.uint8, device=DEV)
    a["dims"] = (T, H, I, K, E, KIND[kind])
    a["kind"] = kind
    return a


def _run_layer(a, probs=True, bias=True, stream=None):
    B.ep_moe_layer(a["x"], a["idx"], a["probs"] if probs else None, a["bias"] if bias else None, a["w_in"],
                   a["s_in"], a["w_out"], a["s_out"], *a["dims"], a["out"], a["ws"], a["ws"].numel(), stream)


def _check_layer(a, probs=True, bias=True):
    T, H, I, K, E, _ = a["dims"]
    want, err = R.layer(a["x"], a["idx"], a["probs"] if probs else None, a["bias"] if bias else None, a["w_in"],
                        a["s_in"], a["w_out"], a["s_out"], a["kind"], E, I)
    R.near(a["out"], want, err, torch.bfloat16)


LAYER = [
    # T, K, E, H, I, kind, masked, repeat, probs, bias
    (1, 1, 1, 8, 8, "bf16", 0.0, False, True, False),
    (1, 8, 64, 512, 136, "bf16", 0.0, False, True, True),
    (3, 2, 5, 264, 72, "bf16", 0.3, False, False, True),
    (16, 4, 16, 2048, 256, "bf16", 0.0, True, True, False),
    (17, 6, 8, 1032, 200, "bf16", 0.2, True, True, True),
    (64, 2, 3, 256, 128, "bf16", 0.0, False, True, False),  # 40 and more tokens per expert
    (16, 64, 100, 128, 64, "bf16", 0.1, False, True, True),
    (5, 4, 1024, 128, 40, "bf16", 0.0, False, True, False),
    (128, 8, 1024, 128, 8, "bf16", 0.1, True, True, True),
    (1, 6, 16, 1024, 384, "fp8", 0.0, False, True, False),
    (9, 8, 32, 640, 256, "fp8", 0.2, True, True, True),
    (100, 1, 2, 256, 128, "fp8", 0.0, False, True, False),  # 50 tokens per expert
    (1, 2, 4, 128, 128, "fp4", 0.0, False, True, True),
    (33, 8, 40, 2048, 384, "fp4", 0.1, False, True, False),
    (128, 8, 64, 7168, 512, "fp4", 0.0, False, True, True),
    (128, 8, 4, 256, 128, "fp4", 0.0, True, True, False),  # 250 entries per expert
    # enough units for the kernels that take 64 channels at once
    (24, 4, 64, 1160, 264, "bf16", 0.1, True, True, True),
    (100, 8, 40, 136, 456, "bf16", 0.0, False, True, False),  # 20 entries per expert
    (60, 8, 48, 384, 384, "fp8", 0.2, False, True, True),
    (120, 8, 20, 128, 896, "fp8", 0.0, False, False, False),  # 48 entries per expert
    (40, 4, 64, 640, 256, "fp4", 0.1, True, True, False),
    (4, 2, 64, 4096, 2048, "fp4", 0.0, False, True, False),  # 8 entries, 32 tiles each
    # two row tiles in the second launch, parts of the long axis that end inside a chunk
    (4, 2, 16, 7168, 640, "fp4", 0.0, False, True, True),
    (4, 2, 16, 4480, 640, "fp8", 0.1, False, True, False),
    (3, 2, 8, 4360, 200, "bf16", 0.0, False, True, True),
    (40, 8, 8, 4360, 136, "bf16", 0.1, False, True, False),  # 40 entries per expert
    (40, 8, 8, 4480, 384, "fp8", 0.0, True, True, True),
    (70, 7, 30, 4480, 896, "fp4", 0.2, True, True, False),  # 13 entries per expert
]


@pytest.mark.parametrize("T,K,E,H,I,kind,masked,repeat,probs,bias", LAYER)
def test_layer(T, K, E, H, I, kind, masked, repeat, probs, bias):
    _say(f"[layer] T={T} K={K} E={E} H={H} I={I} {kind} masked={masked} repeat={repeat}")
    a = _layer_case(T, K, E, H, I, kind, masked, repeat)
    _run_layer(a, probs, bias)
    torch.cuda.synchronize()
    _check_layer(a, probs, bias)


@pytest.mark.parametrize("bias", [False, True])
def test_layer_with_every_entry_masked(bias):
    a = _layer_case(5, 2, 8, 256, 64, "bf16")
    a["idx"].fill_(-1)
    _run_layer(a, bias=bias)
    torch.cuda.synchronize()
    want = a["bias"] if bias else torch.zeros_like(a["out"])
    assert torch.equal(a["out"].view(torch.int16), want.view(torch.int16))


def test_layer_some_rows_masked_and_bias_is_out():
    a = _layer_case(20, 4, 8, 512, 64, "bf16")
    a["idx"][3] = -1
    a["idx"][7:12] = 8
    want, err = R.layer(a["x"], a["idx"], a["probs"], a["bias"], a["w_in"], None, a["w_out"], None, "bf16", 8, 64)
    a["out"] = a["bias"].clone()
    B.ep_moe_layer(a["x"], a["idx"], a["probs"], a["out"], a["w_in"], None, a["w_out"], None, *a["dims"],
                   a["out"], a["ws"], a["ws"].numel())
    torch.cuda.synchronize()
    R.near(a["out"], want, err, torch.bfloat16)
    assert torch.equal(a["out"][3], a["bias"][3])


def test_layer_keeps_infinities_and_nan_of_a_token_in_its_row():
    a = _layer_case(6, 2, 4, 256, 64, "bf16")
    clean = a["x"].clone()
    a["x"][1, 5] = NAN
    a["x"][4, 9] = float("inf")
    _run_layer(a)
    torch.cuda.synchronize()
    assert bool(torch.isnan(a["out"][1]).all()) and not bool(torch.isfinite(a["out"][4]).any())
    a["x"] = clean
    keep = [0, 2, 3, 5]
    got = a["out"][keep].clone()
    _run_layer(a)
    torch.cuda.synchronize()
    assert torch.equal(a["out"][keep], got), "other tokens see none of it"


# ------------------------------------------------------------------ ep_swiglu

SWIGLU = [
    # I, counts, A, type
    (128, [1], 1, "bf16"),
    (128, [3, 0, 2], 4, "fp32"),
    (1408, [17, 0, 40, 1], 16, "bf16"),
    (384, [5] * 300, 1, "fp32"),
    (2048, [130, 0, 0, 64, 1, 200], 128, "bf16"),
    (256, [2000, 1, 0, 3000], 32, "bf16"),
]


def _gate_up(cap, I, rows, dtype, gen):
    """Rows over many binades, with groups of zeros and of tiny and huge values; NaN in the padding."""
    v = torch.full((cap, 2 * I), NAN, dtype=dtype, device=DEV)
    for r in rows:
        z = _normal((len(r), 2 * I), gen, 2.0)
        z = z.unflatten(1, (-1, 128)) * torch.exp2(torch.randint(-6, 3, (len(r), 2 * I // 128, 1), generator=gen, device=DEV))
        pick = torch.randint(0, 12, (len(r), 2 * I // 128, 1), generator=gen, device=DEV)
        z = torch.where(pick == 0, 0.0, torch.where(pick == 1, z * 2.0 ** -130, z))
        v[r.start:r.stop] = z.flatten(1).to(dtype)
    return v


@pytest.mark.parametrize("save", [True, False])
@pytest.mark.parametrize("I,counts,A,kind", SWIGLU)
def test_swiglu(I, counts, A, kind, save):
    _say(f"[swiglu] I={I} experts={len(counts)} A={A} {kind} save={save}")
    gen = _gen(6, I, len(counts), A)
    c, o, rows, cap = _spans(counts, A)
    v = _gate_up(cap, I, rows, TYPE[kind], gen)
    h = torch.full((cap, I), -7.0, dtype=TYPE[kind], device=DEV)
    codes = torch.full((cap, 2 * I), 0x55, dtype=torch.uint8, device=DEV)
    scales = torch.full((cap, 2 * I // 128), -3.0, device=DEV)
    B.ep_swiglu(v, c, o, len(counts), cap, I, KIND[kind], h, codes if save else None, scales if save else None)
    torch.cuda.synchronize()
    live = _real(rows, cap)
    z = v[live].double()
    zero = torch.zeros_like(z[:, :I])
    want, err = R.gated(z[:, :I], zero, z[:, I:], zero)
    R.near(h[live], want, err, TYPE[kind])
    assert bool((h[~live] == -7.0).all())
    if save:
        code, scale = R.checkpoint(v[live])
        assert torch.equal(scales[live].double(), scale)
        assert torch.equal(codes[live].view(torch.float8_e4m3fn).double(), code)
    rest = ~live if save else torch.ones_like(live)
    assert bool((codes[rest] == 0x55).all()) and bool((scales[rest] == -3.0).all())


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_checkpoint_at_the_borders(kind):
    """Largest magnitudes on both sides of 448 * 2^p, rounding ties, the smallest and the largest
    finite values, infinities and NaN."""
    I, cap = 128, 24
    gen = _gen(7)
    v = _normal((cap, 2 * I), gen, 1.0, TYPE[kind])
    top = torch.finfo(TYPE[kind]).max
    for i, m in enumerate([1.75, 1.7578125, 1.75 * 2.0 ** -100, 448.0, 450.0, 449.0, top, top / 4, 2.0 ** -126,
                           2.0 ** -120, 2.0 ** -130, 0.0, 1.0, 2.0 ** -117 * 1.75, 3.5, 3.515625]):
        v[i] = v[i].clamp(-1, 1) * (m / 2)
        v[i, 3], v[i, I + 7] = m, -m
    steps = torch.arange(128, device=DEV) * 0.0625 + 1.03125  # ties of e4m3's 0.125 steps and their neighbours
    v[16, :128] = steps.to(TYPE[kind])
    v[17, 5], v[17, 9], v[18, I + 1] = float("inf"), float("-inf"), NAN
    v[19, :I] = NAN
    h = torch.empty(cap, I, dtype=TYPE[kind], device=DEV)
    codes = torch.empty(cap, 2 * I, dtype=torch.uint8, device=DEV)
    scales = torch.empty(cap, 2, device=DEV)
    B.ep_swiglu(v, None, None, 1, cap, I, KIND[kind], h, codes, scales)
    torch.cuda.synchronize()
    code, scale = R.checkpoint(v)
    assert torch.equal(scales.double(), scale)
    got = codes.view(torch.float8_e4m3fn).double()
    assert torch.equal(torch.isnan(got), torch.isnan(code))
    assert torch.equal(torch.nan_to_num(got, nan=0.0), torch.nan_to_num(code, nan=0.0))
    assert bool(torch.isnan(got[17, [5, 9]]).all()) and bool(torch.isnan(got[19, :I]).all())


@pytest.mark.parametrize("with_h", [True, False])
@pytest.mark.parametrize("I,counts,A,kind", SWIGLU)
def test_swiglu_backward(I, counts, A, kind, with_h):
    _say(f"[swiglu_backward] I={I} experts={len(counts)} A={A} {kind} h={with_h}")
    gen = _gen(8, I, len(counts), A)
    c, o, rows, cap = _spans(counts, A)
    live = _real(rows, cap)
    codes = _normal((cap, 2 * I), gen, 1.0).to(torch.float8_e4m3fn).view(torch.uint8)
    codes[~live] = 0x7F
    scales = torch.rand(cap, 2 * I // 128, generator=gen, device=DEV) * 3  # any scales, not only powers of two
    dh = torch.full((cap, I), NAN, dtype=TYPE[kind], device=DEV)
    dh[live] = _normal((int(live.sum()), I), gen, 0.1, TYPE[kind])
    d = torch.full((cap, 2 * I), -7.0, dtype=TYPE[kind], device=DEV)
    h = torch.full((cap, I), -7.0, dtype=TYPE[kind], device=DEV)
    B.ep_swiglu_backward(dh, codes, scales, c, o, len(counts), cap, I, KIND[kind], d, h if with_h else None)
    torch.cuda.synchronize()
    v = R.values(codes, scales, "fp8")[live].float().double()  # code * scale is one binary32 rounding
    g, u = v[:, :I], v[:, I:]
    want, err = R.gated_backward(dh[live].double(), g, u)
    R.near(d[live], want, err, TYPE[kind])
    zero = torch.zeros_like(g)
    want, err = R.gated(g, zero, u, zero)
    if with_h:
        R.near(h[live], want, err, TYPE[kind])
    assert bool((d[~live] == -7.0).all()) and bool((h[~live] == -7.0).all())
    assert with_h or bool((h == -7.0).all())


def test_swiglu_backward_writes_h_over_dh():
    gen = _gen(9)
    I, cap = 256, 30
    codes = _normal((cap, 2 * I), gen).to(torch.float8_e4m3fn).view(torch.uint8)
    scales = torch.ones(cap, 4, device=DEV)
    dh = _normal((cap, I), gen, 0.1, torch.bfloat16)
    d = [torch.empty(cap, 2 * I, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    h = torch.empty_like(dh)
    B.ep_swiglu_backward(dh, codes, scales, None, None, 1, cap, I, B.EP_BF16, d[0], h)
    B.ep_swiglu_backward(dh, codes, scales, None, None, 1, cap, I, B.EP_BF16, d[1], dh)
    torch.cuda.synchronize()
    assert torch.equal(d[0], d[1]) and torch.equal(h, dh)


def test_swiglu_gradient_against_differences():
    """The backward pass of values that the checkpoint holds exactly, against central differences
    of the forward definition in 64 bits: their error is step^2 / 6 times the third derivative,
    below 2 of the product's size here, and 64-bit rounding."""
    gen = _gen(10)
    I, cap, step = 128, 16, 2.0 ** -14
    codes = _normal((cap, 2 * I), gen, 1.0).to(torch.float8_e4m3fn)
    v = codes.double()
    dh = _normal((cap, I), gen)
    d = torch.empty(cap, 2 * I, device=DEV)
    B.ep_swiglu_backward(dh, codes.view(torch.uint8), torch.ones(cap, 2, device=DEV), None, None, 1, cap, I,
                         B.EP_FP32, d)
    torch.cuda.synchronize()

    def f(z):
        return z[:, :I] * torch.sigmoid(z[:, :I]) * z[:, I:]
    for _ in range(4):
        way = torch.randn(cap, 2 * I, generator=gen, device=DEV, dtype=torch.float64)
        diff = ((f(v + step * way) - f(v - step * way)) / (2 * step) * dh.double()).sum(1)
        got = (d.double() * way).sum(1)
        size = (dh.double().abs() * (1 + v.abs()[:, :I]) * (1 + v.abs()[:, I:]) * (1 + way.abs()[:, :I]) ** 3
                * (1 + way.abs()[:, I:])).sum(1)
        assert bool(((diff - got).abs() <= (2 * step ** 2 + 64 * R.U) * size).all())


# ------------------------------------------------------------------ ep_expert_wgrad

WGRAD = [
    # x kind, H, N, counts, A, dw type, previous, scales
    ("bf16", 8, 8, [1], 1, "fp32", False, False),
    ("bf16", 256, 520, [0, 1, 31, 32, 33, 0, 7], 1, "bf16", False, False),
    ("bf16", 136, 72, [70, 3], 8, "fp32", True, False),
    ("bf16", 1040, 264, [100, 0, 257], 16, "bf16", True, False),
    ("fp8", 128, 128, [64], 1, "fp32", False, True),
    ("fp8", 384, 200, [5, 0, 130, 32], 128, "bf16", False, True),
    ("fp8", 640, 136, [65, 1], 4, "fp32", True, True),
    ("fp8", 48, 24, [9, 40], 1, "fp32", False, False),
    ("fp8", 2048, 1024, [300, 17, 0], 32, "bf16", True, True),
]


def _wgrad_case(kind, H, N, counts, A, grad, previous, scaled, pow2=True, seed=0):
    gen = _gen(11, H, N, len(counts), seed)
    c, o, rows, cap = _spans(counts, A)
    live = _real(rows, cap)
    dy = torch.full((cap, N), NAN, dtype=torch.bfloat16, device=DEV)
    dy[live] = _normal((int(live.sum()), N), gen, 0.1, torch.bfloat16)
    s = None
    if kind == "fp8":
        x = torch.full((cap, H), 0x7F, dtype=torch.uint8, device=DEV)
        x[live] = _normal((int(live.sum()), H), gen, 2.0).to(torch.float8_e4m3fn).view(torch.uint8)
        if scaled:
            s = torch.exp2(torch.randint(-5, 4, (cap, H // 128), generator=gen, device=DEV).float())
            if not pow2:
                s = s * 1.37
            s[~live] = NAN
    else:
        x = torch.full((cap, H), NAN, dtype=torch.bfloat16, device=DEV)
        x[live] = _normal((int(live.sum()), H), gen, 1.0, torch.bfloat16)
    E = len(counts)
    prev = _normal((E, N, H), gen, 1.0, TYPE[grad]) if previous else None
    dw = torch.full((E, N, H), NAN, dtype=TYPE[grad], device=DEV)
    return dict(dy=dy, x=x, s=s, c=c, o=o, rows=rows, cap=cap, prev=prev, dw=dw, E=E, N=N, H=H, kind=kind, grad=grad)


def _run_wgrad(a, stream=None):
    B.ep_expert_wgrad(a["dy"], a["x"], a["s"], a["c"], a["o"], a["E"], a["cap"], a["N"], a["H"], KIND[a["kind"]],
                      a["prev"], a["dw"], KIND[a["grad"]], stream)


def _check_wgrad(a, prev=None):
    prev = a["prev"] if prev is None else prev
    for e, r in enumerate(a["rows"]):
        dy = a["dy"][r.start:r.stop].double()
        x = R.values(a["x"][r.start:r.stop], None if a["s"] is None else a["s"][r.start:r.stop], a["kind"])
        x = x.float().to(torch.bfloat16).double()  # as the definition rounds it
        want, size = dy.T @ x, dy.abs().T @ x.abs()
        if prev is not None:
            want, size = want + prev[e].double(), size + prev[e].double().abs()
        R.near(a["dw"][e], want, (len(r) + 9) * R.U * size, TYPE[a["grad"]])


@pytest.mark.parametrize("kind,H,N,counts,A,grad,previous,scaled", WGRAD)
def test_wgrad(kind, H, N, counts, A, grad, previous, scaled):
    _say(f"[wgrad] {kind} H={H} N={N} counts={counts} A={A} {grad} previous={previous} scaled={scaled}")
    a = _wgrad_case(kind, H, N, counts, A, grad, previous, scaled)
    _run_wgrad(a)
    torch.cuda.synchronize()
    _check_wgrad(a)


def test_wgrad_scales_that_are_no_powers_of_two():
    a = _wgrad_case("fp8", 256, 136, [40, 70], 1, "fp32", False, True, pow2=False)
    _run_wgrad(a)
    torch.cuda.synchronize()
    _check_wgrad(a)


def test_wgrad_scales_of_every_kind_side_by_side():
    """Powers of two inside and outside the range that converts directly, zeros, negative scales,
    subnormal ones and ordinary ones, in rows of one step."""
    a = _wgrad_case("fp8", 256, 136, [40, 70], 1, "fp32", False, True)
    kinds = torch.tensor([1.0, 2.0 ** -70, 0.0, -2.0, 0.75, 2.0 ** 66, -0.0, 2.0 ** -130, 2.0 ** 64, 2.0 ** -64], device=DEV)
    a["s"][:] = kinds[torch.arange(a["s"].numel(), device=DEV) % 10].view_as(a["s"])
    _run_wgrad(a)
    torch.cuda.synchronize()
    _check_wgrad(a)


@pytest.mark.parametrize("grad", ["bf16", "fp32"])
def test_wgrad_accumulates_in_place(grad):
    a = _wgrad_case("bf16", 264, 136, [40, 0, 3], 1, grad, True, False)
    before = a["prev"].clone()
    a["dw"] = a["prev"]
    _run_wgrad(a)
    torch.cuda.synchronize()
    _check_wgrad(a, before)
    assert torch.equal(a["dw"][1], before[1]), "an expert without rows keeps its gradient"


def test_wgrad_of_no_rows_is_zero():
    dw = torch.full((2, 16, 32), NAN, device=DEV)
    none = torch.zeros(3, dtype=torch.int32, device=DEV)
    B.ep_expert_wgrad(None, None, None, none[:2], none, 2, 0, 16, 32, B.EP_BF16, None, dw, B.EP_FP32)
    torch.cuda.synchronize()
    assert bool((dw == 0).all())


# ------------------------------------------------- caps, streams, graphs, together

def _cases_of_all():
    """(name, call, outputs): one call of every operator with its outputs."""
    lay = _layer_case(40, 4, 12, 512, 128, "fp8", 0.1)
    gen = _gen(12)
    counts, A, I = [33, 0, 70, 5], 8, 256
    c, o, rows, cap = _spans(counts, A)
    w, s = _weights(4, 200, 384, "fp4", gen)
    x = _normal((cap, 384), gen, 1.0, torch.bfloat16)
    y = torch.zeros(cap, 200, device=DEV)
    v = _normal((cap, 2 * I), gen, 1.0, torch.bfloat16)
    h = torch.zeros(cap, I, dtype=torch.bfloat16, device=DEV)
    codes = torch.zeros(cap, 2 * I, dtype=torch.uint8, device=DEV)
    scales = torch.zeros(cap, 2 * I // 128, device=DEV)
    d, h2 = torch.zeros_like(v), torch.zeros_like(h)
    wg = _wgrad_case("fp8", 384, 200, counts, A, "fp32", False, True)
    keep = codes.clone(), scales.clone()
    B.ep_swiglu(v, c, o, 4, cap, I, B.EP_BF16, h, *keep)
    torch.cuda.synchronize()
    wide = _layer_case(24, 4, 64, 392, 264, "bf16", 0.1)
    full = _layer_case(128, 8, 64, 7168, 128, "fp4")  # 1024 entries: the most LDS of the second launch
    many = [9, 0, 40, 17] * 10
    mc, mo, _, mcap = _spans(many, 1)
    mw, ms = _weights(40, 904, 384, "fp8", gen)
    mx = _normal((mcap, 384), gen, 1.0, torch.bfloat16)
    my = torch.zeros(mcap, 904, dtype=torch.bfloat16, device=DEV)
    return [
        ("wide layer", lambda st: _run_layer(wide, stream=st), [wide["out"]]),
        ("full layer", lambda st: _run_layer(full, stream=st), [full["out"]]),
        ("wide matvec", lambda st: B.ep_expert_matvec(mx, mw, ms, mc, mo, 40, mcap, 384, 904, B.EP_FP8_E4M3, my, B.EP_BF16, st), [my]),
        ("layer", lambda st: _run_layer(lay, stream=st), [lay["out"]]),
        ("matvec", lambda st: B.ep_expert_matvec(x, w, s, c, o, 4, cap, 384, 200, B.EP_FP4X2, y, B.EP_FP32, st), [y]),
        ("swiglu", lambda st: B.ep_swiglu(v, c, o, 4, cap, I, B.EP_BF16, h, codes, scales, st), [h, codes, scales]),
        ("backward", lambda st: B.ep_swiglu_backward(h, *keep, c, o, 4, cap, I, B.EP_BF16, d, h2, st), [d, h2]),
        ("wgrad", lambda st: _run_wgrad(wg, st), [wg["dw"]]),
    ]


def _bits(ts):
    return [t.clone().view(torch.uint8) for t in ts]


@pytest.mark.parametrize("cap", [1, 3, 64])
def test_results_are_the_same_under_a_workgroup_cap(cap):
    st = torch.cuda.Stream()
    for name, call, outs in _cases_of_all():
        _say(f"[cap {cap}] {name}")
        call(None)
        torch.cuda.synchronize()
        want = _bits(outs)
        for t in outs:
            t.zero_()
        torch.cuda.synchronize()
        try:
            B.ep_set_workgroup_limit(st, cap)
            call(st)
            st.synchronize()
        finally:
            B.ep_set_workgroup_limit(st, 0)
        assert all(torch.equal(a, b) for a, b in zip(want, _bits(outs))), name


def test_captured_calls_replay_with_the_eager_results():
    for name, call, outs in _cases_of_all():
        _say(f"[graph] {name}")
        call(None)
        torch.cuda.synchronize()
        want = _bits(outs)
        st = torch.cuda.Stream()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            call(torch.cuda.current_stream())
        for _ in range(3):
            for t in outs:
                t.zero_()
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, _bits(outs))), name
            call(None)  # the program's own eager call between replays
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, _bits(outs))), name


def test_one_workspace_serves_calls_in_order():
    """A larger call leaves its lists behind; a smaller one on the same stream must not see them."""
    a, b = _layer_case(100, 8, 64, 256, 128, "bf16", seed=3), _layer_case(3, 2, 64, 256, 128, "bf16", seed=4)
    b["idx"][1] = -1
    b["ws"] = a["ws"]
    for _ in range(3):
        _run_layer(a)
        _run_layer(b)
    torch.cuda.synchronize()
    _check_layer(a)
    _check_layer(b)


def test_two_streams_at_once_with_their_own_workspaces():
    a, b = (_layer_case(30, 4, 16, 1024, 256, "bf16", seed=s) for s in (1, 2))
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        _run_layer(a, stream=sa)
        _run_layer(b, stream=sb)
    torch.cuda.synchronize()
    _check_layer(a)
    _check_layer(b)


@pytest.mark.parametrize("T,kind", [(1, "bf16"), (37, "fp8"), (128, "fp4")])
def test_the_layer_is_its_parts(T, kind):
    """layout + dispatch, product, activation, product and combine give what ep_moe_layer gives, to
    the roundings of the rows in between (z, h and y once to bf16 each: half a step of each passed on)."""
    K, E, H, I, A = 4, 24, 512, 256, 1
    a = _layer_case(T, K, E, H, I, kind, 0.1)
    cap = T * K + E * (A - 1)
    i32 = dict(dtype=torch.int32, device=DEV)
    counts, offsets, n = torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(1, **i32)
    dst, meta = torch.empty(T, K, **i32), torch.empty(T, K + 2, **i32)
    wsb = B.ep_layout_dispatch_workspace_bytes(T, K, E)
    ws = torch.empty(max(wsb, 16), dtype=torch.uint8, device=DEV)
    bf = dict(dtype=torch.bfloat16, device=DEV)
    X, Z, Hh, Y = torch.empty(cap, H, **bf), torch.empty(cap, 2 * I, **bf), torch.empty(cap, I, **bf), torch.zeros(cap, H, **bf)
    out = torch.empty(T, H, **bf)
    B.ep_layout_dispatch(a["idx"], T, K, E, A, cap, counts, offsets, dst, meta, n, ws, wsb, a["x"], None, None, H,
                         B.EP_BF16, X, None, None)
    B.ep_expert_matvec(X, a["w_in"], a["s_in"], counts, offsets, E, cap, H, 2 * I, KIND[kind], Z, B.EP_BF16)
    B.ep_swiglu(Z, counts, offsets, E, cap, I, B.EP_BF16, Hh)
    B.ep_expert_matvec(Hh, a["w_out"], a["s_out"], counts, offsets, E, cap, I, H, KIND[kind], Y, B.EP_BF16)
    B.ep_combine(Y, a["probs"], None, dst, T, H, K, B.EP_BF16, cap, out)
    _run_layer(a, bias=False)
    torch.cuda.synchronize()
    _check_layer(a, bias=False)
    half = 2.0 ** -8
    want = torch.zeros(T, H, dtype=torch.float64, device=DEV)
    err = torch.zeros_like(want)
    for t in range(T):
        for k in range(K):
            e = int(a["idx"][t, k])
            if not 0 <= e < E:
                continue
            x = a["x"][t:t + 1].double()
            z, dz = R.product(x, torch.zeros_like(x), R.values(a["w_in"][e], None if a["s_in"] is None else a["s_in"][e], kind))
            dz = dz + half * z.abs()
            h, dh = R.gated(z[:, :I], dz[:, :I], z[:, I:], dz[:, I:])
            y, dy = R.product(h, dh + half * h.abs(), R.values(a["w_out"][e], None if a["s_out"] is None else a["s_out"][e], kind))
            p = float(a["probs"][t, k])
            want[t] += p * y[0]
            err[t] += p * (dy[0] + (half + 8 * R.U) * (y[0].abs() + dy[0]))
    R.near(out, want, err, torch.bfloat16)


def test_training_chain_on_eight_bit_rows():
    """dispatch of 8-bit rows, the activation with its checkpoint, its backward pass and both weight
    gradients, on one layout: every step against its 64-bit form on the inputs it was given."""
    T, K, E, H, I, A = 200, 4, 8, 512, 128, 16
    gen = _gen(13)
    cap = T * K + E * (A - 1)
    idx = _route(T, K, E, 0.05, False, gen)
    x8 = _normal((T, H), gen, 2.0).to(torch.float8_e4m3fn).view(torch.uint8)
    xs = torch.exp2(torch.randint(-4, 2, (T, H // 128), generator=gen, device=DEV).float())
    i32 = dict(dtype=torch.int32, device=DEV)
    counts, offsets, n = torch.empty(E, **i32), torch.empty(E + 1, **i32), torch.empty(1, **i32)
    dst, meta = torch.empty(T, K, **i32), torch.empty(T, K + 2, **i32)
    wsb = B.ep_layout_workspace_bytes(T, K, E)
    ws = torch.empty(max(wsb, 16), dtype=torch.uint8, device=DEV)
    X = torch.zeros(cap, H, dtype=torch.uint8, device=DEV)
    Xs = torch.zeros(cap, H // 128, device=DEV)
    B.ep_layout(idx, T, K, E, A, cap, counts, offsets, dst, meta, n, ws, wsb)
    B.ep_dispatch(x8, xs, None, dst, T, H, K, B.EP_FP8_E4M3, cap, X, Xs, None)
    bf = dict(dtype=torch.bfloat16, device=DEV)
    Z, dH, dY = _normal((cap, 2 * I), gen, 1.0, torch.bfloat16), _normal((cap, I), gen, 0.1, torch.bfloat16), _normal((cap, H), gen, 0.1, torch.bfloat16)
    Hh, codes, scales = torch.zeros(cap, I, **bf), torch.zeros(cap, 2 * I, dtype=torch.uint8, device=DEV), torch.zeros(cap, 2, device=DEV)
    dZ, H2 = torch.zeros(cap, 2 * I, **bf), torch.zeros(cap, I, **bf)
    dWin, dWout = torch.empty(E, 2 * I, H, device=DEV), torch.empty(E, H, I, device=DEV)
    B.ep_swiglu(Z, counts, offsets, E, cap, I, B.EP_BF16, Hh, codes, scales)
    B.ep_swiglu_backward(dH, codes, scales, counts, offsets, E, cap, I, B.EP_BF16, dZ, H2)
    B.ep_expert_wgrad(dZ, X, Xs, counts, offsets, E, cap, 2 * I, H, B.EP_FP8_E4M3, None, dWin, B.EP_FP32)
    B.ep_expert_wgrad(dY, H2, None, counts, offsets, E, cap, H, I, B.EP_BF16, None, dWout, B.EP_FP32)
    torch.cuda.synchronize()
    rows = [range(int(offsets[e]), int(offsets[e]) + int(counts[e])) for e in range(E)]
    live = _real(rows, cap)
    v = R.values(codes, scales, "fp8")[live]
    code, scale = R.checkpoint(Z[live])
    assert torch.equal(scales[live].double(), scale)
    assert torch.equal(codes[live].view(torch.float8_e4m3fn).double(), code)
    want, err = R.gated_backward(dH[live].double(), v[:, :I], v[:, I:])
    R.near(dZ[live], want, err, torch.bfloat16)
    # 16 of 256 steps of e4m3 at most: the checkpoint's values are within half a step of the rows
    step = scale.repeat_interleave(128, -1)
    assert bool(((v - Z[live].double()).abs() <= torch.maximum(2.0 ** -4 * Z[live].double().abs(), 2.0 ** -10 * step)).all())
    common = dict(c=counts, o=offsets, rows=rows, cap=cap, prev=None, E=E, grad="fp32")
    _check_wgrad(dict(common, dy=dZ, x=X, s=Xs, dw=dWin, N=2 * I, H=H, kind="fp8"))
    _check_wgrad(dict(common, dy=dY, x=H2, s=None, dw=dWout, N=H, H=I, kind="bf16"))


def test_rows_and_matrices_behind_four_gib():
    """Rows at the end of buffers of more than 2^32 bytes, and the last expert's matrix of more
    than 2^32 bytes of them: every offset that passes 32 bits is taken in 64."""
    gen = _gen(14)
    cap, K, N, n = 300_000, 8192, 256, 5
    c = torch.tensor([0, n], dtype=torch.int32, device=DEV)
    o = torch.tensor([0, cap - n, cap], dtype=torch.int32, device=DEV)
    x = torch.empty(cap, K, dtype=torch.bfloat16, device=DEV)
    x[-n:] = _normal((n, K), gen, 1.0, torch.bfloat16)
    w, _ = _weights(2, N, K, "bf16", gen)
    y = torch.empty(cap, N, device=DEV)
    B.ep_expert_matvec(x, w, None, c, o, 2, cap, K, N, B.EP_BF16, y, B.EP_FP32)
    h = torch.empty(cap, K // 2, dtype=torch.bfloat16, device=DEV)
    codes = torch.empty(cap, K, dtype=torch.uint8, device=DEV)
    scales = torch.empty(cap, K // 128, device=DEV)
    B.ep_swiglu(x, c, o, 2, cap, K // 2, B.EP_BF16, h, codes, scales)
    d = torch.empty_like(x)
    B.ep_swiglu_backward(h, codes, scales, c, o, 2, cap, K // 2, B.EP_BF16, d)
    dw = torch.empty(2, N, K, device=DEV)
    dy = torch.empty(cap, N, dtype=torch.bfloat16, device=DEV)
    dy[-n:] = _normal((n, N), gen, 1.0, torch.bfloat16)
    B.ep_expert_wgrad(dy, x, None, c, o, 2, cap, N, K, B.EP_BF16, None, dw, B.EP_FP32)
    torch.cuda.synchronize()
    z = x[-n:].double()
    want, err = R.product(z, torch.zeros_like(z), w[1].double())
    R.near(y[-n:], want, err, torch.float32)
    half = K // 2
    zero = torch.zeros_like(z[:, :half])
    want, err = R.gated(z[:, :half], zero, z[:, half:], zero)
    R.near(h[-n:], want, err, torch.bfloat16)
    code, scale = R.checkpoint(x[-n:])
    assert torch.equal(scales[-n:].double(), scale)
    assert torch.equal(codes[-n:].view(torch.float8_e4m3fn).double(), code)
    v = R.values(codes[-n:], scales[-n:], "fp8")
    want, err = R.gated_backward(h[-n:].double(), v[:, :half], v[:, half:])
    R.near(d[-n:], want, err, torch.bfloat16)
    a = dy[-n:].double()
    assert bool((dw[0] == 0).all())
    R.near(dw[1], a.T @ z, (n + 9) * R.U * (a.abs().T @ z.abs()), torch.float32)
    del x, y, h, codes, d, dw, dy
    # the gradient and the weights of 40 experts: 4.7 GB each
    E, N, H, n = 40, 4096, 7168, 3
    counts = [0] * (E - 1) + [n]
    c, o, _, cap = _spans(counts, 1)
    x = _normal((cap, H), gen, 1.0, torch.bfloat16)
    dy = _normal((cap, N), gen, 1.0, torch.bfloat16)
    dw = torch.full((E, N, H), NAN, device=DEV)
    B.ep_expert_wgrad(dy, x, None, c, o, E, cap, N, H, B.EP_BF16, None, dw, B.EP_FP32)
    w = torch.empty(2 * E, N, H, dtype=torch.bfloat16, device=DEV)
    w[-1] = _normal((N, H), gen, H ** -0.5, torch.bfloat16)
    y = torch.empty(cap, N, device=DEV)
    B.ep_expert_matvec(x, w, None, torch.cat([torch.zeros(E, dtype=torch.int32, device=DEV), c]),
                       torch.cat([torch.zeros(E, dtype=torch.int32, device=DEV), o]), 2 * E, cap, H, N, B.EP_BF16, y,
                       B.EP_FP32)
    torch.cuda.synchronize()
    a, z = dy.double(), x.double()
    R.near(dw[-1], a.T @ z, (n + 9) * R.U * (a.abs().T @ z.abs()), torch.float32)
    assert bool((dw[:-1] == 0).all())
    want, err = R.product(z, torch.zeros_like(z), w[-1].double())
    R.near(y, want, err, torch.float32)
