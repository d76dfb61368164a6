"""binary32 logits that hold bf16 values, as a projection in bf16 and a cast leave them: many are equal.

Ids are those of the same logits in bf16, ties by the lowest id, also where three to six equal logits meet at the last
place.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - only on CPU hosts
    pytest.skip("needs a GPU", allow_module_level=True)

from tests.test_gpu_router import DEV, Forward, _backward, _gen  # noqa: E402


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,K", [(6000, 64, 6), (4000, 256, 8), (1000, 256, 16), (2000, 1024, 8)])
def test_logits_cast_from_bf16(T, E, K, scoring):
    print(f"[bf16 values] T={T} E={E} K={K} {scoring}", flush=True)
    gen = _gen(51, T, E)
    l = (torch.randn(T, E, generator=gen, device=DEV) * 1.5).bfloat16()
    f = Forward(l.float(), K, scoring)().check()
    g = Forward(l, K, scoring)().check()
    assert torch.equal(f.idx, g.idx) and torch.equal(f.counts, g.counts)
    _backward(f, torch.randn(T, K, generator=gen, device=DEV), 0.5, None)
    Forward(l.float(), K, scoring, bias=torch.zeros(E, device=DEV))().check()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,K", [(20, 4), (256, 8), (256, 14), (1000, 8)])
def test_equal_logits_at_the_last_place(E, K, scoring):
    print(f"[last place] E={E} K={K} {scoring}", flush=True)
    gen = _gen(52, E, K)
    T = 240
    l = torch.randn(T, E, generator=gen, device=DEV).clamp(max=1.5).bfloat16().float()
    for n in range(T):
        at = torch.randperm(E, generator=gen, device=DEV)
        equal = 3 + n % 4
        above = max(0, K - 1 - n // 4 % equal)  # the K-th place is one of the equal ones
        l[n, at[:above]] = 4.0 + torch.arange(above, device=DEV)
        l[n, at[above:above + equal]] = 3.0
    Forward(l, K, scoring)().check()
    Forward(l, K, scoring, bias=torch.zeros(E, device=DEV))().check()
    Forward(l, K, scoring, bias=torch.full((E,), 0.25, device=DEV))().check()
