"""Refusals of the experts' operators: every check runs on the host before anything is enqueued (no
GPU needed), and the 64-bit forms that the GPU tests compare with, on their own."""
import os

import pytest

from combine_ep_layout_amd import binding as B

FAKE = 1 << 20  # a 16-byte aligned, never dereferenced address
ODD = FAKE + 4  # misaligned for rows


@pytest.fixture(scope="module", autouse=True)
def L():
    if not os.path.exists(B.LIB_PATH):
        from combine_ep_layout_amd import build
        build.build()
    return B.lib()


def _code(fn, *a):
    with pytest.raises(B.EpError) as ei:
        fn(*a)
    assert B.ep_last_error().startswith(fn.__name__ + ":")
    return ei.value.code


def layer(**kw):
    a = dict(x=FAKE, idx=FAKE, w=None, bias=None, w_in=FAKE, s_in=None, w_out=FAKE, s_out=None, T=8, H=512, I=256,
             K=2, E=4, dt=B.EP_BF16, out=FAKE, ws=FAKE, wsb=1 << 20)
    a.update(kw)
    return tuple(a.values())


LAYER = [dict(T=-1), dict(K=0), dict(K=65), dict(E=0), dict(E=1025), dict(H=0), dict(H=7), dict(H=516), dict(I=0),
         dict(I=12), dict(dt=B.EP_FP32), dict(dt=9), dict(s_in=FAKE), dict(s_out=FAKE), dict(x=None), dict(idx=None),
         dict(out=None), dict(ws=None), dict(w_in=None), dict(w_out=None), dict(x=ODD), dict(out=ODD), dict(bias=ODD),
         dict(ws=ODD), dict(w_in=ODD), dict(w_out=ODD), dict(idx=FAKE + 2), dict(w=FAKE + 1), dict(wsb=1000),
         dict(dt=B.EP_FP8_E4M3), dict(dt=B.EP_FP8_E4M3, s_in=FAKE), dict(dt=B.EP_FP4X2, s_in=FAKE, s_out=FAKE, H=576),
         dict(dt=B.EP_FP8_E4M3, s_in=FAKE, s_out=FAKE, I=192), dict(dt=B.EP_FP4X2, s_in=FAKE, s_out=FAKE + 2),
         dict(H=1 << 20, I=1 << 10)]


@pytest.mark.parametrize("kw", LAYER, ids=str)
def test_layer_refusals(kw):
    assert _code(B.ep_moe_layer, *layer(**kw)) == B.EP_EINVAL


def test_layer_of_too_many_entries():
    assert _code(B.ep_moe_layer, *layer(T=129, K=8)) == B.EP_EUNSUPPORTED
    assert _code(B.ep_moe_layer, *layer(T=1 << 30, K=1)) == B.EP_EUNSUPPORTED


def test_layer_of_no_tokens_launches_nothing():
    B.ep_moe_layer(*layer(T=0, x=None, idx=None, out=None, ws=None, wsb=0))


def test_layer_workspace():
    assert B.ep_moe_layer_workspace_bytes(0, 8, 256) == 0
    assert B.ep_moe_layer_workspace_bytes(129, 8, 256) == 0
    assert B.ep_moe_layer_workspace_bytes(-1, 8, 256) == 0
    assert B.ep_moe_layer_workspace_bytes(1, 8, 0) == 0
    for T, K, I in [(1, 1, 8), (3, 7, 72), (128, 8, 2048), (16, 64, 128)]:
        n = T * K
        assert 4 * n * I + 6 * n <= B.ep_moe_layer_workspace_bytes(T, K, I) <= 4 * n * I + 6 * n + 512


def matvec(**kw):
    a = dict(x=FAKE, w=FAKE, s=None, c=FAKE, o=FAKE, E=4, cap=64, K=512, N=256, dt=B.EP_BF16, y=FAKE, yd=B.EP_BF16)
    a.update(kw)
    return tuple(a.values())


MATVEC = [dict(E=0), dict(E=1025), dict(cap=-1), dict(cap=1 << 31), dict(c=None), dict(o=None), dict(c=None, o=None),
          dict(c=FAKE + 1), dict(o=FAKE + 2), dict(K=0), dict(K=12), dict(N=0), dict(N=12), dict(dt=B.EP_FP32),
          dict(yd=B.EP_FP8_E4M3), dict(yd=7), dict(s=FAKE), dict(dt=B.EP_FP4X2), dict(dt=B.EP_FP4X2, s=FAKE, K=192),
          dict(x=None), dict(y=None), dict(w=None), dict(x=ODD), dict(y=ODD), dict(w=ODD), dict(K=1 << 20, N=1 << 12)]


@pytest.mark.parametrize("kw", MATVEC, ids=str)
def test_matvec_refusals(kw):
    assert _code(B.ep_expert_matvec, *matvec(**kw)) == B.EP_EINVAL


def test_matvec_of_no_rows_launches_nothing():
    B.ep_expert_matvec(*matvec(cap=0, x=None, y=None))


FAR = 1 << 24  # beyond the rows of the other operands below


def swiglu(**kw):
    a = dict(v=FAKE, c=FAKE, o=FAKE, E=4, cap=64, I=256, dt=B.EP_BF16, h=FAKE + FAR, codes=FAKE, s=FAKE)
    a.update(kw)
    return tuple(a.values())


SWIGLU = [dict(E=0), dict(cap=-1), dict(c=None), dict(c=None, o=None), dict(I=0), dict(I=192), dict(I=-128),
          dict(I=12, codes=None, s=None), dict(dt=B.EP_FP8_E4M3), dict(codes=None), dict(s=None), dict(v=None),
          dict(h=None), dict(v=ODD), dict(h=FAKE + FAR + 8), dict(codes=ODD), dict(s=FAKE + 2), dict(h=FAKE),
          dict(h=FAKE + 64 * 512 * 2 - 16), dict(I=1 << 25)]


@pytest.mark.parametrize("kw", SWIGLU, ids=str)
def test_swiglu_refusals(kw):
    assert _code(B.ep_swiglu, *swiglu(**kw)) == B.EP_EINVAL


def backward(**kw):
    a = dict(dh=FAKE, codes=FAKE, s=FAKE, c=FAKE, o=FAKE, E=4, cap=64, I=256, dt=B.EP_BF16, d=FAKE + FAR, h=None)
    a.update(kw)
    return tuple(a.values())


BACKWARD = [dict(E=1025), dict(cap=-1), dict(o=None), dict(I=192), dict(dt=B.EP_FP4X2), dict(codes=None), dict(s=None),
            dict(dh=None), dict(d=None), dict(dh=ODD), dict(d=FAKE + FAR + 8), dict(h=FAKE + 2 * FAR + 8), dict(d=FAKE),
            dict(h=FAKE + FAR), dict(h=FAKE + 16)]


@pytest.mark.parametrize("kw", BACKWARD, ids=str)
def test_swiglu_backward_refusals(kw):
    assert _code(B.ep_swiglu_backward, *backward(**kw)) == B.EP_EINVAL


def test_swiglu_of_no_rows_launches_nothing():
    B.ep_swiglu(*swiglu(cap=0, v=None, h=None))
    B.ep_swiglu_backward(*backward(cap=0, dh=None, codes=None, s=None, d=None))


def wgrad(**kw):
    a = dict(dy=FAKE, x=FAKE, s=None, c=FAKE, o=FAKE, E=4, cap=64, N=256, H=512, xd=B.EP_BF16, prev=None, dw=FAKE,
             dd=B.EP_BF16)
    a.update(kw)
    return tuple(a.values())


WGRAD = [dict(E=0), dict(cap=-1), dict(c=None), dict(c=None, o=None), dict(N=0), dict(N=12), dict(H=0), dict(H=12),
         dict(H=24, xd=B.EP_FP8_E4M3), dict(H=192, xd=B.EP_FP8_E4M3, s=FAKE), dict(s=FAKE), dict(xd=B.EP_FP32),
         dict(xd=B.EP_FP4X2), dict(dd=B.EP_FP8_E4M3), dict(dy=None), dict(x=None), dict(dw=None), dict(dy=ODD),
         dict(x=ODD), dict(dw=ODD), dict(prev=ODD), dict(prev=FAKE + 16), dict(xd=B.EP_FP8_E4M3, s=FAKE + 2)]


@pytest.mark.parametrize("kw", WGRAD, ids=str)
def test_wgrad_refusals(kw):
    assert _code(B.ep_expert_wgrad, *wgrad(**kw)) == B.EP_EINVAL


def test_the_64_bit_forms_on_known_values():
    torch = pytest.importorskip("torch")
    from tests import experts_ref as R
    # e2m1 pairs: the low half is the value of even index
    assert R.codes_e2m1(torch.tensor([[0x10, 0x7F, 0x9A]], dtype=torch.uint8)).tolist() == [[0.0, 0.5, -6.0, 6.0, -1.0, -0.5]]
    v = torch.zeros(1, 256)
    v[0, 0], v[0, 1], v[0, 2], v[0, 128] = 448.0, 17.0, 19.0, 449.0
    code, scale = R.checkpoint(v)
    assert scale.tolist() == [[1.0, 2.0]]
    assert code[0, :3].tolist() == [448.0, 16.0, 20.0] and code[0, 128] == 224.0  # ties to even
    # against torch's own conversion, over every binade of e4m3
    g = torch.randn(64, 128, generator=torch.Generator().manual_seed(1)) * 2.0 ** torch.arange(-32, 32).view(64, 1) / 8
    code, scale = R.checkpoint(g)
    assert torch.equal(code, (g.double() / scale.repeat_interleave(128, -1)).float().to(torch.float8_e4m3fn).double())
    d, _ = R.gated_backward(torch.ones(1, 1, dtype=torch.float64), torch.zeros(1, 1, dtype=torch.float64),
                            torch.full((1, 1), 3.0, dtype=torch.float64))
    assert d.tolist() == [[1.5, 0.0]]
