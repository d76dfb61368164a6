"""Weight gradients from 8-bit rows with scales of any kind, against products that are not rounded.

The bound: code * scale is rounded once to binary32 (2^-24 of it, or 2^-150 where it is subnormal) and
kept to 24 bits; what lies below 2^-133, the least step of bf16, is cut. Sums as in experts_ref: a sum of
n binary32 products within (n + 8) * 2^-23 of the sum of their magnitudes, here of up to three parts a row.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - only on CPU hosts
    pytest.skip("needs a GPU", allow_module_level=True)

from combine_ep_layout_amd import binding as B  # noqa: E402
from tests import experts_ref as R  # noqa: E402

DEV = "cuda:0"
KIND = {torch.float32: B.EP_FP32, torch.bfloat16: B.EP_BF16}


def _case(counts, N, H, seed, A=1):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    off = [0]
    for n in counts:
        off.append(off[-1] + -(-n // A) * A)
    cap = off[-1]
    i32 = dict(dtype=torch.int32, device=DEV)
    dy = torch.randn(cap, N, generator=gen, device=DEV).mul_(0.1).bfloat16()
    x = torch.randn(cap, H, generator=gen, device=DEV).mul_(2.0).to(torch.float8_e4m3fn).view(torch.uint8)
    s = torch.rand(cap, H // 128, generator=gen, device=DEV) * 0.99 + 0.01
    return dict(c=torch.tensor(counts, **i32), o=torch.tensor(off, **i32), off=off, counts=counts, cap=cap, dy=dy, x=x,
                s=s, N=N, H=H, gen=gen)


def _run(a, prev=None, dtype=torch.float32, stream=None):
    dw = torch.full((len(a["counts"]), a["N"], a["H"]), float("nan"), dtype=dtype, device=DEV)
    B.ep_expert_wgrad(a["dy"], a["x"], a["s"], a["c"], a["o"], len(a["counts"]), a["cap"], a["N"], a["H"],
                      B.EP_FP8_E4M3, prev, dw, KIND[dtype], stream)
    torch.cuda.synchronize()
    return dw


def _check(a, dw, prev=None):
    for e, n in enumerate(a["counts"]):
        r = slice(a["off"][e], a["off"][e] + n)
        dy, x = a["dy"][r].double(), R.values(a["x"][r], a["s"][r], "fp8")
        want, size = dy.T @ x, dy.abs().T @ x.abs()
        if prev is not None:
            want, size = want + prev[e].double(), size + prev[e].double().abs()
        cut = dy.abs().sum(0)[:, None] * 2.0 ** -133
        R.near(dw[e], want, (3 * n + 9) * R.U * size + cut, dw.dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("previous", [False, True])
@pytest.mark.parametrize("counts,N,H", [([1], 8, 128), ([40, 0, 70], 136, 256), ([31, 32, 33, 130], 264, 384),
                                        ([300, 5], 72, 640)])
def test_scales_as_dispatch_moves_them(counts, N, H, previous, dtype):
    print(f"[wgrad scales] {counts} N={N} H={H} previous={previous} {dtype}", flush=True)
    a = _case(counts, N, H, 1)
    prev = torch.randn(len(counts), N, H, generator=a["gen"], device=DEV).to(dtype) if previous else None
    _check(a, _run(a, prev, dtype), prev)


def test_error_is_that_of_a_sum_in_binary32():
    """128 rows with scales in [0.01, 1]: relative to the gradient's size, root mean square. Rounding x to
    bf16 would give about 2^-9 / sqrt(3) = 1.1e-3; a sum in binary32 stays below 128 * 2^-24 = 7.7e-6."""
    a = _case([128], 256, 512, 2)
    got = _run(a)[0].double()
    want = a["dy"].double().T @ R.values(a["x"], a["s"], "fp8")
    assert float((got - want).norm() / want.norm()) < 128 * 2.0 ** -24


@pytest.mark.parametrize("where", ["first row", "last row", "row 32", "row 95", "one group", "second group"])
def test_one_inexact_scale_among_powers_of_two(where):
    """Wherever it stands, a scale that needs more bits is kept whole, and the other experts' tiles too."""
    a = _case([5, 130, 64], 200, 384, 3)
    a["s"] = torch.exp2(torch.randint(-5, 4, a["s"].shape, generator=a["gen"], device=DEV).float())
    first = a["off"][1]
    row = {"first row": 0, "last row": 129, "row 32": 32, "row 95": 95}.get(where)
    if row is not None:
        a["s"][first + row] *= 1.37
    else:
        a["s"][first:first + 130, 0 if where == "one group" else 1] *= 1.37
    _check(a, _run(a))


def test_results_do_not_depend_on_the_cap_or_the_call():
    a = _case([5, 130, 64, 0, 33], 264, 640, 4)
    a["s"][5:135] = torch.exp2(torch.round(torch.log2(a["s"][5:135])))  # one expert converts directly
    want = _run(a)
    _check(a, want)
    st = torch.cuda.Stream()
    for cap in (1, 2, 7):
        B.ep_set_workgroup_limit(st, cap)
        try:
            assert torch.equal(_run(a, stream=st), want)
        finally:
            B.ep_set_workgroup_limit(st, 0)
    assert torch.equal(_run(a), want)
    dw = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=st):
        B.ep_expert_wgrad(a["dy"], a["x"], a["s"], a["c"], a["o"], 5, a["cap"], 264, 640, B.EP_FP8_E4M3, None, dw,
                          B.EP_FP32, torch.cuda.current_stream())
    for _ in range(3):
        dw.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(dw, want)


def test_scales_at_the_ends_of_binary32():
    """Products near the largest value, and down to subnormal ones next to each other in a column's rows."""
    for top in (2.0 ** 118 * 1.37, 2.0 ** -100 * 1.37, 2.0 ** -118 * 1.37, 2.0 ** -126, 2.0 ** -126 * 1.37):
        a = _case([50], 64, 256, 5)
        a["s"].fill_(top)
        if top < 1:
            a["dy"] = (a["dy"].float() * 2.0 ** 100).bfloat16()
        _check(a, _run(a))


@pytest.mark.parametrize("bad", [float("inf"), float("-inf"), float("nan"), "code"])
def test_infinite_and_nan_values_stay_in_their_columns(bad):
    a = _case([40, 33], 72, 384, 6)
    clean = _run(a)
    if bad == "code":
        a["x"][45, 130] = 0x7F
        hit = torch.zeros(384, dtype=torch.bool, device=DEV)
        hit[130] = True
    else:
        a["s"][45, 1] = bad
        hit = torch.zeros(384, dtype=torch.bool, device=DEV)
        hit[128:256] = True
    got = _run(a)
    assert torch.equal(got[0], clean[0]) and torch.equal(got[1][:, ~hit], clean[1][:, ~hit])
    x = R.values(a["x"][40:73], a["s"][40:73], "fp8")[:, hit]
    want = a["dy"][40:73].double().T @ x
    # a sum with one infinite term is that infinity, with a NaN it is NaN (0 * infinity among them)
    assert torch.equal(torch.isnan(got[1][:, hit]), torch.isnan(want))
    inf = torch.isinf(want)
    assert torch.equal(got[1][:, hit][inf].double(), want[inf])


def test_zero_scales_and_zero_rows():
    a = _case([70], 72, 256, 7)
    a["x"][33:50] = 0
    a["s"][33:50] = 2.0 ** -126
    a["s"][10], a["s"][11] = 0.0, -0.0
    a["x"][60, 3] = 0x80
    _check(a, _run(a))
