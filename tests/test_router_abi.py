"""Refusals of the router's and the 8-bit integer operators (every check runs on the host before anything
is enqueued: no GPU needed), their workspace, and the 64-bit forms that the GPU tests compare with."""
import os

import pytest

from combine_ep_layout_amd import binding as B

FAKE = 1 << 20  # a 16-byte aligned, never dereferenced address
ODD = FAKE + 4  # misaligned for rows
FAR = 1 << 34   # beyond the rows of the other operands below


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


def router(**kw):
    a = dict(l=FAKE, bias=None, mask=None, seq=None, T=8, E=16, K=2, S=1, dt=B.EP_FP32, sc=B.EP_SOFTMAX, norm=1, scale=1.0,
             given=0, idx=FAKE, w=FAKE, c=FAKE, n=FAKE, b=FAKE, z=FAKE, ws=FAKE, wsb=1 << 20)
    a.update(kw)
    return tuple(a.values())


ROUTER = [dict(T=-1), dict(K=0), dict(K=65, E=128), dict(E=0), dict(E=1025), dict(K=17), dict(S=0), dict(S=2), dict(S=1 << 17, seq=FAKE),
          dict(dt=B.EP_FP8_E4M3), dict(dt=7), dict(sc=2), dict(sc=-1), dict(scale=float("nan")), dict(scale=float("inf")),
          dict(given=1, bias=FAKE), dict(given=1, mask=FAKE), dict(c=None), dict(n=None), dict(c=None, n=None),
          dict(c=None, n=None, z=None), dict(sc=B.EP_SIGMOID), dict(l=None), dict(idx=None), dict(l=ODD), dict(ws=ODD),
          dict(ws=None), dict(wsb=16), dict(idx=FAKE + 2), dict(w=FAKE + 1), dict(bias=FAKE + 2), dict(seq=FAKE + 1, S=1),
          dict(c=FAKE + 2), dict(n=FAKE + 2), dict(b=FAKE + 2), dict(z=FAKE + 2), dict(T=1 << 30, K=4), dict(T=2 ** 31 - 1, K=1)]


@pytest.mark.parametrize("kw", ROUTER, ids=str)
def test_router_refusals(kw):
    assert _code(B.ep_router, *router(**kw)) == B.EP_EINVAL


def backward(**kw):
    a = dict(l=FAKE, idx=FAKE, seq=None, c=FAKE, n=FAKE, dw=FAKE, db=FAKE, dz=FAKE, T=8, E=16, K=2, S=1, dt=B.EP_FP32,
             sc=B.EP_SOFTMAX, norm=1, scale=1.0, d=FAKE + FAR)
    a.update(kw)
    return tuple(a.values())


BACKWARD = [dict(T=-1), dict(T=2 ** 31 - 1, K=1), dict(K=0), dict(K=65), dict(E=0), dict(E=1025), dict(S=0), dict(S=3), dict(dt=B.EP_FP4X2), dict(sc=5),
            dict(scale=float("nan")), dict(c=None), dict(n=None), dict(c=None, n=None), dict(c=None, n=None, db=None),
            dict(sc=B.EP_SIGMOID), dict(l=None), dict(idx=None), dict(d=None), dict(l=ODD), dict(d=FAKE + FAR + 4), dict(d=FAKE),
            dict(d=FAKE + 16), dict(idx=FAKE + 2), dict(dw=FAKE + 2), dict(db=FAKE + 1), dict(dz=FAKE + 2), dict(seq=FAKE + 2)]


@pytest.mark.parametrize("kw", BACKWARD, ids=str)
def test_router_backward_refusals(kw):
    assert _code(B.ep_router_backward, *backward(**kw)) == B.EP_EINVAL


def test_router_of_no_tokens_launches_nothing():
    B.ep_router(*router(T=0, l=None, idx=None, w=None, c=None, n=None, b=None, z=None, ws=None, wsb=0))
    B.ep_router_backward(*backward(T=0, l=None, idx=None, d=None))


def test_router_workspace():
    size = B.ep_router_workspace_bytes
    assert size(-1, 16, 1) == 0 and size(4, 0, 1) == 0 and size(4, 1025, 1) == 0 and size(4, 16, 0) == 0
    assert size(4, 16, (1 << 16) + 1) == 0
    assert 0 < size(0, 16, 1) <= 1024
    for T, E, S in [(1, 1, 1), (4096, 256, 1), (4096, 256, 300), (100000, 1024, 7)]:
        # a sum and a count per expert for every tile of tokens and every sequence, at most one tile in 16 tokens;
        # for every sequence its terms of the losses, at most one for four experts
        assert size(T, E, S) <= (T // 16 + 1 + S) * (8 * E + 8) + S * (8 * (E // 4 + 1) + 8) + 128
        assert size(2 * T, E, S) >= size(T, E, S) and size(T, E, S + 1) >= size(T, E, S)


def quantize(**kw):
    a = dict(x=FAKE, c=FAKE, o=FAKE, E=4, cap=64, W=256, dt=B.EP_BF16, codes=FAKE + FAR, s=FAKE, cols=1)
    a.update(kw)
    return tuple(a.values())


QUANTIZE = [dict(E=0), dict(E=1025), dict(cap=-1), dict(cap=1 << 31), dict(c=None), dict(o=None), dict(c=None, o=None), dict(W=0),
            dict(W=8), dict(W=200), dict(W=(1 << 24) + 16), dict(dt=B.EP_FP8_E4M3), dict(dt=9), dict(cols=0), dict(cols=(1 << 20) + 1),
            dict(x=None), dict(codes=None), dict(s=None), dict(x=ODD), dict(codes=FAKE + FAR + 8), dict(s=FAKE + 2), dict(codes=FAKE),
            dict(codes=FAKE + 64 * 512 - 16), dict(c=FAKE + 1), dict(o=FAKE + 2)]


@pytest.mark.parametrize("fn", [B.ep_quantize_rows, B.ep_swiglu_quantize], ids=lambda f: f.__name__)
@pytest.mark.parametrize("kw", QUANTIZE, ids=str)
def test_quantize_refusals(fn, kw):
    assert _code(fn, *quantize(**kw)) == B.EP_EINVAL


def test_quantize_of_no_rows_launches_nothing():
    for fn in (B.ep_quantize_rows, B.ep_swiglu_quantize):
        fn(*quantize(cap=0, x=None, codes=None, s=None))


def matmul(**kw):
    a = dict(x=FAKE, s=FAKE, cols=1, w=FAKE, ws=FAKE, c=FAKE, o=FAKE, E=4, cap=64, K=512, N=256, y=FAKE, yd=B.EP_BF16)
    a.update(kw)
    return tuple(a.values())


MATMUL = [dict(E=0), dict(E=1025), dict(cap=-1), dict(cap=1 << 31), dict(c=None), dict(o=None), dict(c=None, o=None), dict(K=0),
          dict(K=8), dict(K=200), dict(K=131072), dict(N=0), dict(N=12), dict(N=(1 << 23) + 8), dict(K=65536, N=32768), dict(cols=0),
          dict(cols=1 << 21), dict(yd=B.EP_FP8_E4M3), dict(yd=5), dict(x=None), dict(s=None), dict(w=None), dict(ws=None), dict(y=None),
          dict(x=ODD), dict(w=ODD), dict(y=ODD), dict(s=FAKE + 2), dict(ws=FAKE + 1), dict(c=FAKE + 2)]


@pytest.mark.parametrize("kw", MATMUL, ids=str)
def test_matmul_refusals(kw):
    assert _code(B.ep_quantized_matmul, *matmul(**kw)) == B.EP_EINVAL


def test_matmul_of_no_rows_launches_nothing():
    B.ep_quantized_matmul(*matmul(cap=0, x=None, s=None, y=None))


def test_the_widest_sum_fits():
    assert 128 * 128 * B.EP_MAX_QUANTIZED_WIDTH < 2 ** 31 <= 128 * 128 * (B.EP_MAX_QUANTIZED_WIDTH + 16)


# ------------------------------------------------------------------ the 64-bit forms on their own

def test_the_router_forms_on_known_values():
    torch = pytest.importorskip("torch")
    from tests import router_ref as R
    l = torch.tensor([[0.0, 1.0, 1.0, -R.INF], [2.0, 2.0, -R.INF, -R.INF]], dtype=torch.float64)
    ids = R.choose(l, 3, "softmax")
    assert ids.tolist() == [[1, 2, 0], [0, 1, -1]]  # ties by id, -infinity never
    w, _ = R.weights(l, ids, "softmax", True, 2.0)
    assert w[1].tolist() == [1.0, 1.0, 0.0]
    assert R.choose(l, 1, "sigmoid", bias=torch.tensor([0.5, 0.0, 0.0, 9.0])).tolist() == [[0], [0]]
    assert R.choose(l, 2, "softmax", mask=torch.tensor([0, 1])).tolist() == [[-1, -1], [0, 1]]
    # even use of the experts has balance 1, one expert for all E
    flat = torch.zeros(4, 4, dtype=torch.float64)
    _, tokens, (balance, _), (z, _) = R.statistics(flat, torch.arange(4)[:, None], "softmax", None)
    assert abs(balance - 1) < 1e-12 and tokens.tolist() == [4, 1, 4] and abs(z - torch.log(torch.tensor(4.0)) ** 2) < 1e-6
    sharp = torch.tensor([[99.0, 0, 0, 0]] * 4, dtype=torch.float64)
    assert abs(R.statistics(sharp, torch.zeros(4, 1, dtype=torch.long), "softmax", None)[2][0] - 4) < 1e-9


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [False, True])
def test_the_gradient_formulas_against_differences(scoring, normalize):
    """The formulas of the backward pass against central differences of the forward forms, in 64 bits."""
    torch = pytest.importorskip("torch")
    from tests import router_ref as R
    gen = torch.Generator().manual_seed(5)
    T, E, K, scale = 7, 6, 3, 1.7
    l = torch.randn(T, E, generator=gen, dtype=torch.float64)
    ids = torch.randint(-1, E, (T, K), generator=gen)  # some masked, some twice
    ids[3] = -1
    dw = torch.randn(T, K, generator=gen, dtype=torch.float64)
    seq = torch.tensor([1, 3, 3, 6])
    db, dz = 0.7, 0.3 if scoring == "softmax" else None
    counts, tokens, _, _ = R.statistics(l, ids, scoring, seq)

    def value(x):
        w, _ = R.weights(x, ids, scoring, normalize, scale)
        _, _, (balance, _), (z, _) = R.statistics(x, ids, scoring, seq)
        return float((w * dw).sum()) + db * balance + (dz or 0.0) * z

    d, _ = R.backward(l, ids, scoring, normalize, scale, dw, seq, counts, tokens, db, dz)
    h = 1e-5
    for t in range(T):
        for e in range(E):
            x = l.clone()
            x[t, e] += h
            y = l.clone()
            y[t, e] -= h
            assert abs((value(x) - value(y)) / (2 * h) - float(d[t, e])) < 1e-8  # h^2 and 1e-16 / h
