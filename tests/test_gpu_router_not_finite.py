"""Rows with NaN or +infinity among their logits: which experts are chosen, and that no other row notices.

A NaN logit leaves its own expert out and no other, with and without a bias. Of scores + bias, the scores are those of
the row without its NaN logits; experts at +infinity share a probability of 1 (a sigmoid of 1 each).
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
NAN, INF = float("nan"), float("inf")


def _choose(l, K, scoring, bias):
    """In 64 bits, row by row in plain words."""
    nan, top = torch.isnan(l), l == INF
    if bias is None:
        key = l
    else:
        score = torch.sigmoid(l)
        if scoring == "softmax":
            score = torch.softmax(torch.where(nan, -INF, l), 1)
            share = top / top.sum(1, keepdim=True).clamp(min=1).double()
            score = torch.where(top.any(1, keepdim=True), share, score)
        key = torch.where(l == -INF, -INF, score + bias.double())
    key = torch.where(nan | torch.isnan(key), -INF, key)
    v, ids = torch.sort(key, dim=1, descending=True, stable=True)
    return torch.where(v[:, :K] == -INF, -1, ids[:, :K])


def _call(l, kind, K, scoring, bias, normalize):
    T, E = l.shape
    idx, w = torch.full((T, K), -7, dtype=torch.int32, device=DEV), torch.full((T, K), -7.0, device=DEV)
    B.ep_router(l, bias, None, None, T, E, K, 1, KIND[kind], SCORING[scoring], int(normalize), 2.0, 0, idx, w)
    torch.cuda.synchronize()
    return idx.long(), w


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [True, False])
@pytest.mark.parametrize("E,K,kind", [(12, 4, "fp32"), (100, 8, "bf16"), (256, 8, "fp32"), (256, 20, "fp32"), (600, 8, "bf16"), (1000, 62, "fp32")])
def test_a_nan_or_infinite_logit(E, K, kind, biased, scoring):
    print(f"[not finite] E={E} K={K} {kind} biased={biased} {scoring}", flush=True)
    gen = torch.Generator(device=DEV).manual_seed(E * 64 + K)
    clean = (torch.randn(40, E, generator=gen, device=DEV) * 1.5).to(TYPE[kind])
    bias = torch.randn(E, generator=gen, device=DEV) * 0.1 if biased else None
    l = clean.clone()
    l[1, 3] = NAN
    l[2, E - 1] = INF
    l[3, [2, 9]] = INF
    l[5, 4], l[5, 6] = NAN, INF
    l[6] = NAN
    l[7, 1:] = NAN
    l[9, :E // 2] = NAN
    l[10] = INF
    l[11] = -INF
    l[11, 5] = NAN
    l[12], l[12, 7], l[12, 8] = -INF, NAN, 0.5
    broken = torch.zeros(40, dtype=torch.bool, device=DEV)
    broken[[1, 2, 3, 5, 6, 7, 9, 10, 11, 12]] = True
    for normalize in (True, False):
        ids, w = _call(l, kind, K, scoring, bias, normalize)
        want = _choose(l.double(), K, scoring, bias)
        assert torch.equal(ids, want), f"rows {torch.nonzero((ids != want).any(1)).flatten().tolist()}"
        there, whole = _call(clean, kind, K, scoring, bias, normalize)
        assert torch.equal(ids[~broken], there[~broken]) and torch.equal(w[~broken], whole[~broken])
        assert bool((w[ids < 0] == 0).all())
    # normalised weights depend on the chosen logits alone, so NaN among the others leaves them whole
    _, w = _call(l, kind, K, scoring, bias, True)
    rows = [1, 7, 9, 12]
    exact, err = R.weights(torch.where(torch.isnan(l), -INF, l)[rows].double(), want[rows], scoring, True, 2.0)
    R.near(w[rows], exact, err, torch.float32)
