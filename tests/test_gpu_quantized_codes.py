"""Every code, and every value between two codes, at a factor that is a power of two: nothing is rounded but the code.

With a row's largest magnitude 127 * 2^p, the scale is 2^p and the factor 2^-p. All rows looked at are real ones.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - only on CPU hosts
    pytest.skip("needs a GPU", allow_module_level=True)

from combine_ep_layout_amd import binding as B  # noqa: E402

DEV = "cuda:0"
KIND = {"bf16": B.EP_BF16, "fp32": B.EP_FP32}
TYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}
POWERS = [-100, -93, -40, -7, -1, 0, 1, 30, 110, 120]


def _rows(W):
    """(values, codes) of rows that go through -127 .. 127 by halves; halves go to the even code."""
    k = torch.arange(W, device=DEV) % 509 - 254  # in halves
    rows, codes = [], []
    for start in range(0, 509, 73):
        v = torch.roll(k, start)
        v[start % W] = 254  # the largest, wherever it is
        low = torch.div(v, 2, rounding_mode="floor")
        rows.append(v / 2)
        codes.append(torch.where(v % 2 == 0, low, low + low % 2))
    return torch.stack(rows), torch.stack(codes).to(torch.int8)


def _spans(n):
    """n rows of two experts among padding: (counts, offsets, the rows' places, rows of the buffer)."""
    first = n // 2
    at = torch.cat([torch.arange(first), 64 + torch.arange(n - first)]).to(DEV)
    return (torch.tensor([first, n - first], dtype=torch.int32, device=DEV), torch.tensor([0, 64, 128], dtype=torch.int32, device=DEV),
            at, 128)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("W", [512, 1040, 7168, 40000])
def test_every_code(W, kind):
    print(f"[codes] W={W} {kind}", flush=True)
    v, want = _rows(W)
    assert want.unique().numel() >= 254
    c, o, at, cap = _spans(len(v))
    for p in POWERS:
        x = torch.full((cap, W), float("nan"), dtype=TYPE[kind], device=DEV)
        x[at] = (v.double() * 2.0 ** p).to(TYPE[kind])
        assert torch.equal(x[at].double(), v.double() * 2.0 ** p), "the values are exact"
        codes, scales = torch.full((cap, W), 99, dtype=torch.int8, device=DEV), torch.full((cap, 1), -7.0, device=DEV)
        B.ep_quantize_rows(x, c, o, 2, cap, W, KIND[kind], codes, scales, 1)
        torch.cuda.synchronize()
        assert torch.equal(codes[at], want) and bool((scales[at] == 2.0 ** p).all()), p


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("W", [512, 2064])
def test_every_code_of_the_activation(W, kind):
    """A gate of 128 is its own activation: exp(-128) is lost beside 1."""
    print(f"[gated codes] W={W} {kind}", flush=True)
    v, want = _rows(W)
    c, o, at, cap = _spans(len(v))
    for p in (-90, -40, 0, 30, 110):
        x = torch.full((cap, 2 * W), float("nan"), dtype=TYPE[kind], device=DEV)
        x[at, :W] = 128.0
        x[at, W:] = (v.double() * 2.0 ** (p - 7)).to(TYPE[kind])
        codes, scales = torch.full((cap, W), 99, dtype=torch.int8, device=DEV), torch.full((cap, 1), -7.0, device=DEV)
        B.ep_swiglu_quantize(x, c, o, 2, cap, W, KIND[kind], codes, scales, 1)
        torch.cuda.synchronize()
        assert torch.equal(codes[at], want) and bool((scales[at] == 2.0 ** p).all()), p
