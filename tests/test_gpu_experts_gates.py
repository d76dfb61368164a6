"""The gated activation at gates where exp(-gate) or its reciprocal leaves binary32's normal numbers.

At a gate of -87.4 the sigmoid is below 2^-126 and at -88.8 exp(-gate) passes the largest binary32 value,
while gate * sigmoid(gate) * up is still a normal number for a large up. The bounds are experts_ref's:
(|gate| + 8) * 2^-23 relative, and binary32's least step where a result is subnormal.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - only on CPU hosts
    pytest.skip("needs a GPU", allow_module_level=True)

from combine_ep_layout_amd import binding as B  # noqa: E402
from tests import experts_ref as R  # noqa: E402

DEV = "cuda:0"
TYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}
KIND = {"bf16": B.EP_BF16, "fp32": B.EP_FP32}
GATES = [-80.0, -86.0, -87.0, -87.5, -88.0, -88.5, -89.0, -90.0, -96.0, -100.0, -104.0, -120.0, -150.0, -200.0, -1e4, -1e30,
         0.0, 88.0, 90.0, 200.0, 1e4, -1.0]
UPS = [1.0, -4.0, 1e-3, 1e10, -1e20, 1e30, 3e38, 0.0]


def _rows(kind):
    """Every gate with every up, eight channels of a group apart, the rest ordinary values."""
    gen = torch.Generator(device=DEV).manual_seed(1)
    v = torch.randn(len(GATES), 256, generator=gen, device=DEV)
    for i, g in enumerate(GATES):
        for j, u in enumerate(UPS):
            v[i, 5 + 13 * j], v[i, 128 + 5 + 13 * j] = g, u
    return v.to(TYPE[kind])


@pytest.mark.parametrize("save", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_forward(kind, save):
    v = _rows(kind)
    n = v.shape[0]
    h = torch.empty(n, 128, dtype=TYPE[kind], device=DEV)
    codes = torch.empty(n, 256, dtype=torch.uint8, device=DEV) if save else None
    scales = torch.empty(n, 2, device=DEV) if save else None
    B.ep_swiglu(v, None, None, 1, n, 128, KIND[kind], h, codes, scales)
    torch.cuda.synchronize()
    z = v.double()
    zero = torch.zeros_like(z[:, :128])
    want, err = R.gated(z[:, :128], zero, z[:, 128:], zero)
    fits = want.abs() < torch.finfo(TYPE[kind]).max * 0.99
    assert bool(torch.isinf(h[want.abs() > torch.finfo(torch.float32).max * 1.01]).all())
    R.near(torch.where(fits, h, 0), torch.where(fits, want, 0.0), torch.where(fits, err, 0.0), TYPE[kind])


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_forward_of_infinities_and_nan(kind):
    inf, nan = float("inf"), float("nan")
    cases = [(inf, 1.0, inf), (inf, -2.0, -inf), (inf, 0.0, nan), (-inf, 1.0, nan), (nan, 1.0, nan), (1.0, nan, nan),
             (1.0, inf, inf), (-1.0, inf, -inf), (-1.0, -inf, inf), (0.0, inf, nan), (-89.0, nan, nan)]
    v = torch.ones(1, 256, dtype=TYPE[kind], device=DEV)
    for i, (g, u, _) in enumerate(cases):
        v[0, i], v[0, 128 + i] = g, u
    h = torch.empty(1, 128, dtype=TYPE[kind], device=DEV)
    B.ep_swiglu(v, None, None, 1, 1, 128, KIND[kind], h)
    torch.cuda.synchronize()
    want = torch.tensor([c[2] for c in cases])
    got = h[0, :len(cases)].float().cpu()
    assert torch.equal(torch.isnan(got), torch.isnan(want)), got
    assert torch.equal(got[~torch.isnan(want)], want[~torch.isnan(want)]), got
    assert bool((h[0, len(cases):].double() - 0.7310585786300049).abs().max() < 2.0 ** -8)


@pytest.mark.parametrize("with_h", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "fp32"])
def test_backward(kind, with_h):
    """Gates as the checkpoint gives them: codes of -1.75, -1.375 and the like times 2^6, and scales
    that are no powers of two."""
    I, n = 128, 12
    gen = torch.Generator(device=DEV).manual_seed(2)
    codes = torch.randn(n, 2 * I, generator=gen, device=DEV).clamp(-2, 2).to(torch.float8_e4m3fn)
    codes[:, :64] = torch.tensor([-1.25, -1.375, -1.5, -1.625, -1.75, -1.875, -2.0, 1.5], device=DEV).repeat(8).to(codes.dtype)
    scales = torch.empty(n, 2, device=DEV)
    scales[:, 0] = torch.tensor([64.0, 63.5, 65.0, 70.0, 50.0, 47.0, 90.0, 1000.0, 1e30, 1.0, 46.0, 54.5], device=DEV)
    scales[:, 1] = torch.tensor([1.0, 1e10, 1e20, 1e30, 1e37, 1e25, 1e30, 1.0, 1.0, 1e10, 1e30, 1e38], device=DEV)
    dh = torch.randn(n, I, generator=gen, device=DEV).to(TYPE[kind])
    dh[:, ::3] *= 2.0 ** 100 if kind == "fp32" else 2.0 ** 96
    d = torch.empty(n, 2 * I, dtype=TYPE[kind], device=DEV)
    h = torch.empty(n, I, dtype=TYPE[kind], device=DEV) if with_h else None
    B.ep_swiglu_backward(dh, codes.view(torch.uint8), scales, None, None, 1, n, I, KIND[kind], d, h)
    torch.cuda.synchronize()
    v = R.values(codes.view(torch.uint8), scales, "fp8").float().double()
    g, u = v[:, :I], v[:, I:]
    want, err = R.gated_backward(dh.double(), g, u)
    # a few binary32 roundings of results that may be subnormal, scaled by what multiplies them after
    x = dh.double().abs()
    err = err + 2.0 ** -148 * torch.cat([(x + u.abs() + 1) * (1 + g.abs()), (x + 1) * (1 + g.abs())], 1)
    top = torch.finfo(TYPE[kind]).max
    # where no factor pair passes the largest value on the way, whatever the order
    size = torch.cat([(x + 1) * (u.abs() + 1) * (1 + g.abs()), (x + 1) * (1 + g.abs()).expand_as(x)], 1)
    fits = size < top * 0.5
    assert int(fits.sum()) > fits.numel() // 2
    R.near(torch.where(fits, d, 0), torch.where(fits, want, 0.0), torch.where(fits, err, 0.0), TYPE[kind])
    if with_h:
        zero = torch.zeros_like(g)
        want, err = R.gated(g, zero, u, zero)
        fits = (u.abs() + 1) * (g.abs() + 1) < top * 0.5
        R.near(torch.where(fits, h, 0), torch.where(fits, want, 0.0), torch.where(fits, err, 0.0), TYPE[kind])


@pytest.mark.parametrize("E", [1, 300])  # 16 channels a workgroup, and 64
def test_layer(E):
    """A layer whose gates and ups are its weights (one token of a single one), passed on by w_out."""
    H, I = 8, 64
    T = 1 if E == 1 else 300
    g = torch.tensor((GATES * 3)[:I], device=DEV)
    u = torch.tensor((UPS * 8)[:I], device=DEV).roll(3)
    x = torch.zeros(T, H, dtype=torch.bfloat16, device=DEV)
    x[:, 0] = 1
    w_in = torch.zeros(E, 2 * I, H, dtype=torch.bfloat16, device=DEV)
    w_in[:, :I, 0], w_in[:, I:, 0] = g.bfloat16(), u.bfloat16()
    w_out = torch.zeros(E, H, I, dtype=torch.bfloat16, device=DEV)
    for out in range(H):  # one channel of h each: see every gate in turn
        w_out[:, out, out] = 1
    idx = torch.arange(T, dtype=torch.int32, device=DEV)[:, None] % E
    gd, ud = w_in[0, :I, 0].double(), w_in[0, I:, 0].double()
    zero = torch.zeros_like(gd)
    h, err = R.gated(gd, zero, ud, zero)
    ws = torch.empty(B.ep_moe_layer_workspace_bytes(T, 1, I), dtype=torch.uint8, device=DEV)
    out = torch.empty(T, H, dtype=torch.bfloat16, device=DEV)
    for first in range(0, I, H):
        w_out.zero_()
        for c in range(H):
            if h[first + c].abs() < 3e38:
                w_out[:, c, first + c] = 1
        w_now = w_in.clone()
        w_now[:, :I][:, h.abs() >= 3e38] = 0
        B.ep_moe_layer(x, idx, None, None, w_now, None, w_out, None, T, H, I, 1, E, B.EP_BF16, out, ws, ws.numel())
        torch.cuda.synchronize()
        want = torch.where(h.abs() < 3e38, h, 0.0)[first:first + H].expand(T, H)
        # h as two bf16 parts: 2^-17, and bf16's least step
        allowed = (err + 2.0 ** -16 * h.abs() + 2.0 ** -132)[first:first + H].expand(T, H)
        R.near(out, want, torch.where(want == 0, 0.0, allowed), torch.bfloat16)
