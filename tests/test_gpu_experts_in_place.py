"""Outputs in the place of inputs, where the header allows it: the results of separate buffers, bit for bit."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - only on CPU hosts
    pytest.skip("needs a GPU", allow_module_level=True)

from combine_ep_layout_amd import binding as B  # noqa: E402

DEV = "cuda:0"
TYPE = {"bf16": torch.bfloat16, "fp32": torch.float32}
KIND = {"bf16": B.EP_BF16, "fp32": B.EP_FP32}


@pytest.fixture(params=[0, 1, 5], ids=lambda c: f"cap{c}")
def stream(request):
    st = torch.cuda.Stream()
    if request.param:
        B.ep_set_workgroup_limit(st, request.param)
    yield st
    B.ep_set_workgroup_limit(st, 0)


@pytest.mark.parametrize("kind", ["bf16", "fp32"])
@pytest.mark.parametrize("I,counts,A", [(128, [1], 1), (384, [17, 0, 40, 3], 16), (1408, [900, 5, 0, 1300], 32)])
def test_swiglu_backward_h_over_dh(kind, I, counts, A, stream):
    gen = torch.Generator(device=DEV).manual_seed(I)
    off = [0]
    for n in counts:
        off.append(off[-1] + -(-n // A) * A)
    cap, E = off[-1], len(counts)
    i32 = dict(dtype=torch.int32, device=DEV)
    c, o = torch.tensor(counts, **i32), torch.tensor(off, **i32)
    codes = torch.randn(cap, 2 * I, generator=gen, device=DEV).to(torch.float8_e4m3fn).view(torch.uint8)
    scales = torch.rand(cap, 2 * I // 128, generator=gen, device=DEV)
    dh = torch.randn(cap, I, generator=gen, device=DEV).to(TYPE[kind])
    d = [torch.zeros(cap, 2 * I, dtype=TYPE[kind], device=DEV) for _ in range(2)]
    h = dh.clone()  # padding rows keep what the buffer held
    torch.cuda.synchronize()
    B.ep_swiglu_backward(dh, codes, scales, c, o, E, cap, I, KIND[kind], d[0], h, stream)
    B.ep_swiglu_backward(dh, codes, scales, c, o, E, cap, I, KIND[kind], d[1], dh, stream)
    torch.cuda.synchronize()
    assert torch.equal(d[0], d[1]) and torch.equal(h, dh)


@pytest.mark.parametrize("T,K,E,H,I,kind", [(1, 2, 4, 264, 64, "bf16"), (70, 4, 6, 512, 128, "fp8"), (40, 2, 30, 4480, 128, "fp4"),
                                            (60, 8, 8, 4360, 136, "bf16")])
def test_layer_bias_is_out(T, K, E, H, I, kind, stream):
    gen = torch.Generator(device=DEV).manual_seed(T)
    x = torch.randn(T, H, generator=gen, device=DEV).bfloat16()
    idx = torch.randint(-1, E, (T, K), generator=gen, device=DEV, dtype=torch.int32)
    probs = torch.rand(T, K, generator=gen, device=DEV)

    def weights(n, width):
        if kind == "bf16":
            return torch.randn(E, n, width, generator=gen, device=DEV).mul_(width ** -0.5).bfloat16(), None
        w = torch.randint(0, 120, (E, n, width if kind == "fp8" else width // 2), generator=gen, device=DEV, dtype=torch.uint8)
        return w, torch.rand(E, n, width // 128, generator=gen, device=DEV) * 0.01

    (wi, si), (wo, so) = weights(2 * I, H), weights(H, I)
    dt = {"bf16": B.EP_BF16, "fp8": B.EP_FP8_E4M3, "fp4": B.EP_FP4X2}[kind]
    bias = torch.randn(T, H, generator=gen, device=DEV).bfloat16()
    ws = torch.empty(B.ep_moe_layer_workspace_bytes(T, K, I), dtype=torch.uint8, device=DEV)
    out, both = torch.empty_like(bias), bias.clone()
    torch.cuda.synchronize()
    for b, y in ((bias, out), (both, both)):
        B.ep_moe_layer(x, idx, probs, b, wi, si, wo, so, T, H, I, K, E, dt, y, ws, ws.numel(), stream)
    torch.cuda.synchronize()
    assert torch.equal(out.view(torch.int16), both.view(torch.int16))
    assert bool(torch.isfinite(out).all())
