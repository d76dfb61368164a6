"""Given ids that point at excluded experts only (logits of -infinity) in rows that have other logits.

The weights are 0, and nothing flows back through them; the token has ids, so it takes part in counts and losses with
the probabilities and the log sum of its whole row.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - only on CPU hosts
    pytest.skip("needs a GPU", allow_module_level=True)

from tests.test_gpu_router import DEV, Forward, _backward, _gen, _logits  # noqa: E402


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("E,K,kind", [(16, 3, "fp32"), (256, 8, "bf16"), (700, 20, "fp32")])
def test_ids_at_excluded_experts(E, K, kind, normalize, scoring):
    print(f"[excluded] E={E} K={K} {kind} normalize={normalize} {scoring}", flush=True)
    T, gen = 60, _gen(31, E, K)
    l = _logits(T, E, kind, gen)
    out = torch.arange(E, device=DEV) < E // 2
    l[:, out] = -float("inf")
    ids = torch.randint(0, E, (T, K), generator=gen, device=DEV)
    dead = torch.arange(T, device=DEV) % 3 == 0
    ids[dead] = ids[dead] % (E // 2)
    f = Forward(l, K, scoring, normalize, 1.5, ids=ids)().check()
    assert bool((f.w[dead] == 0).all()) and int(f.tokens[0]) == T and int(f.counts.sum()) == T * K
    d = _backward(f, torch.randn(T, K, generator=gen, device=DEV), 0.5, 0.25 if scoring == "softmax" else None)
    assert bool((d[:, out] == 0).all()) and bool((d[dead] != 0).any(1).all())
    only = _backward(f, torch.randn(T, K, generator=gen, device=DEV), None, None)
    assert bool((only[dead] == 0).all())
