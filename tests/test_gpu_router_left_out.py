"""Tokens without ids (masked, or given ids outside the experts) whose logits are garbage.

A padded batch's rows may hold anything. Such a token has weights and a gradient of exactly 0, takes no part in counts
and losses, and leaves the other tokens' results as they are without it.
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
NAN, INF = float("nan"), float("inf")


def _pass(l, kind, K, scoring, normalize, given, out, dw):
    """Forward and backward with both losses; `out`: tokens left out."""
    T, E = l.shape
    soft = scoring == B.EP_SOFTMAX
    idx = torch.full((T, K), -7, dtype=torch.int32, device=DEV)
    if given:
        idx = torch.randint(0, E, (T, K), generator=torch.Generator(device=DEV).manual_seed(3), device=DEV, dtype=torch.int32)
        idx[out] = -1
        idx[out[0], 0] = E
    w = torch.full((T, K), -7.0, device=DEV)
    counts, tokens = torch.empty(1, E, dtype=torch.int32, device=DEV), torch.empty(3, dtype=torch.int32, device=DEV)
    losses = torch.zeros(2, device=DEV)
    mask = torch.ones(T, dtype=torch.uint8, device=DEV)
    mask[out] = 0
    wsb = B.ep_router_workspace_bytes(T, E, 1)
    ws = torch.empty(wsb, dtype=torch.uint8, device=DEV)
    B.ep_router(l, None, None if given else mask, None, T, E, K, 1, KIND[kind], scoring, int(normalize), 1.5, int(given), idx, w,
                counts, tokens, losses, losses[1:] if soft else None, ws, wsb)
    d = torch.full_like(l, -7.0)
    one = torch.full((1,), 0.5, device=DEV)
    B.ep_router_backward(l, idx, None, counts, tokens, dw, one, one if soft else None, T, E, K, 1, KIND[kind], scoring, int(normalize),
                         1.5, d)
    torch.cuda.synchronize()
    return idx, w, counts, tokens, losses, d


@pytest.mark.parametrize("scoring", [B.EP_SOFTMAX, B.EP_SIGMOID], ids=["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("given", [True, False], ids=["given", "masked"])
@pytest.mark.parametrize("E,K,kind", [(64, 6, "bf16"), (256, 8, "fp32"), (50, 20, "fp32"), (600, 8, "bf16")])
def test_tokens_without_ids_have_no_gradient(E, K, kind, given, normalize, scoring):
    print(f"[left out] E={E} K={K} {kind} given={given} normalize={normalize} scoring={scoring}", flush=True)
    T, gen = 70, torch.Generator(device=DEV).manual_seed(E + K)
    clean = (torch.randn(T, E, generator=gen, device=DEV) * 1.5).to(TYPE[kind])
    dw = torch.randn(T, K, generator=gen, device=DEV)
    out = torch.tensor([2, 3, 4, 17, 33, 69], device=DEV)
    broken = clean.clone()
    broken[2] = NAN
    broken[3, 1] = NAN
    broken[4, E - 1] = INF
    broken[17] = INF
    broken[33] = -INF
    broken[69, ::2] = NAN
    want = _pass(clean, kind, K, scoring, normalize, given, out, dw)
    got = _pass(broken, kind, K, scoring, normalize, given, out, dw)
    keep = torch.ones(T, dtype=torch.bool, device=DEV)
    keep[out] = False
    for a, b in zip(got[:2], want[:2]):  # ids and weights
        assert torch.equal(a[keep], b[keep])
    assert bool((got[1][out] == 0).all())
    for a, b in zip(got[2:5], want[2:5]):  # counts, tokens, losses
        assert torch.equal(a, b)
    assert torch.equal(got[5][keep], want[5][keep])
    assert bool((got[5][out] == 0).all()), f"rows {out[(got[5][out] != 0).any(1)].tolist()} have a gradient"
