"""Spans that cross an end of the expand buffer: every operator takes exactly the rows inside."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - only on CPU hosts
    pytest.skip("needs a GPU", allow_module_level=True)

from combine_ep_layout_amd import binding as B  # noqa: E402
from tests import experts_ref as R  # noqa: E402

DEV = "cuda:0"
TOP = (1 << 31) - 1


def _spans(E, cap):
    """Routing arrays whose first span begins before the buffer, whose last one ends behind it, with
    spans that hold nothing or lie outside (their sums pass 32 bits); and the rows inside of each."""
    begin, count = [-3], [8]  # rows 0 to 4
    for e in range(1, E - 1):
        begin.append(5 + 2 * e)
        count.append(e % 3)
    begin += [cap - 4, TOP]  # the last four rows; offsets has one more element
    count += [9]
    if E >= 5:
        begin[2], count[2] = -TOP - 1, TOP  # ends at -1
        begin[3], count[3] = TOP, TOP  # begins behind the buffer
    rows = [range(max(b, 0), max(max(b, 0), min(b + c, cap))) for b, c in zip(begin, count)]
    i32 = dict(dtype=torch.int32, device=DEV)
    return torch.tensor(count, **i32), torch.tensor(begin, **i32), rows


def _inside(rows, cap):
    live = torch.zeros(cap, dtype=torch.bool, device=DEV)
    for r in rows:
        live[r.start:r.stop] = True
    return live


@pytest.mark.parametrize("E,K,N", [(2, 256, 72), (6, 1152, 200), (40, 256, 1024)])  # the last: many tiles
def test_matvec(E, K, N):
    cap = 5 + 2 * E + 8
    c, o, rows = _spans(E, cap)
    gen = torch.Generator(device=DEV).manual_seed(E)
    x = torch.randn(cap, K, generator=gen, device=DEV).bfloat16()
    w = torch.randn(E, N, K, generator=gen, device=DEV).bfloat16()
    y = torch.full((cap, N), -7.0, device=DEV)
    B.ep_expert_matvec(x, w, None, c, o, E, cap, K, N, B.EP_BF16, y, B.EP_FP32)
    torch.cuda.synchronize()
    for e, r in enumerate(rows):
        z = x[r.start:r.stop].double()
        want, err = R.product(z, torch.zeros_like(z), w[e].double())
        if len(r):
            R.near(y[r.start:r.stop], want, err, torch.float32)
    assert bool((y[~_inside(rows, cap)] == -7.0).all())


@pytest.mark.parametrize("kind", ["bf16", "fp8"])
@pytest.mark.parametrize("previous", [False, True])
def test_wgrad(kind, previous):
    E, N, H = 6, 72, 256
    cap = 5 + 2 * E + 8
    c, o, rows = _spans(E, cap)
    gen = torch.Generator(device=DEV).manual_seed(7)
    dy = torch.randn(cap, N, generator=gen, device=DEV).bfloat16()
    x = torch.randn(cap, H, generator=gen, device=DEV)
    x = x.bfloat16() if kind == "bf16" else x.to(torch.float8_e4m3fn).view(torch.uint8)
    prev = torch.randn(E, N, H, generator=gen, device=DEV) if previous else None
    dw = torch.full((E, N, H), float("nan"), device=DEV)
    B.ep_expert_wgrad(dy, x, None, c, o, E, cap, N, H, B.EP_BF16 if kind == "bf16" else B.EP_FP8_E4M3, prev, dw,
                      B.EP_FP32)
    torch.cuda.synchronize()
    for e, r in enumerate(rows):
        a, z = dy[r.start:r.stop].double(), R.values(x[r.start:r.stop], None, kind)
        want, size = a.T @ z, a.abs().T @ z.abs()
        if previous:
            want, size = want + prev[e].double(), size + prev[e].double().abs()
        R.near(dw[e], want, (len(r) + 9) * R.U * size, torch.float32)


def test_swiglu_and_its_backward_pass():
    E, I = 6, 128
    cap = 5 + 2 * E + 8
    c, o, rows = _spans(E, cap)
    live = _inside(rows, cap)
    gen = torch.Generator(device=DEV).manual_seed(8)
    v = torch.randn(cap, 2 * I, generator=gen, device=DEV)
    h = torch.full((cap, I), -7.0, device=DEV)
    codes = torch.full((cap, 2 * I), 0x55, dtype=torch.uint8, device=DEV)
    scales = torch.full((cap, 2), -3.0, device=DEV)
    B.ep_swiglu(v, c, o, E, cap, I, B.EP_FP32, h, codes, scales)
    dh = torch.randn(cap, I, generator=gen, device=DEV)
    d = torch.full((cap, 2 * I), -7.0, device=DEV)
    B.ep_swiglu_backward(dh, codes, scales, c, o, E, cap, I, B.EP_FP32, d)
    torch.cuda.synchronize()
    z = v[live].double()
    zero = torch.zeros_like(z[:, :I])
    want, err = R.gated(z[:, :I], zero, z[:, I:], zero)
    R.near(h[live], want, err, torch.float32)
    code, scale = R.checkpoint(v[live])
    assert torch.equal(scales[live].double(), scale)
    assert torch.equal(codes[live].view(torch.float8_e4m3fn).double(), code)
    z = R.values(codes[live], scales[live], "fp8")
    want, err = R.gated_backward(dh[live].double(), z[:, :I], z[:, I:])
    R.near(d[live], want, err, torch.float32)
    assert bool((h[~live] == -7.0).all()) and bool((codes[~live] == 0x55).all())
    assert bool((scales[~live] == -3.0).all()) and bool((d[~live] == -7.0).all())


def test_no_sum_of_offset_and_count_wraps_into_the_buffer():
    """Sums that 32 bits would wrap round to a few rows: nothing is inside."""
    K, N, cap = 128, 72, 4
    i32 = dict(dtype=torch.int32, device=DEV)
    o = torch.tensor([-TOP - 1, -TOP - 1, TOP, -5, 0, 0], **i32)
    c = torch.tensor([-TOP - 1 + 9, -TOP - 1, TOP, -TOP, -3], **i32)
    x = torch.ones(cap, K, device=DEV).bfloat16()
    w = torch.ones(5, N, K, device=DEV).bfloat16()
    y = torch.full((cap, N), -7.0, device=DEV)
    B.ep_expert_matvec(x, w, None, c, o, 5, cap, K, N, B.EP_BF16, y, B.EP_FP32)
    dw = torch.full((5, N, K), 3.0, device=DEV)
    dy = torch.ones(cap, N, device=DEV).bfloat16()
    B.ep_expert_wgrad(dy, x, None, c, o, 5, cap, N, K, B.EP_BF16, None, dw, B.EP_FP32)
    v = torch.ones(cap, 2 * K, device=DEV)
    h = torch.full((cap, K), -7.0, device=DEV)
    B.ep_swiglu(v, c, o, 5, cap, K, B.EP_FP32, h)
    torch.cuda.synchronize()
    assert bool((y == -7.0).all()) and bool((dw == 0).all()) and bool((h == -7.0).all())
