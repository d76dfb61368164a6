"""One workspace, sized for the largest batch, for batches of every smaller size, experts and sequences alike."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - only on CPU hosts
    pytest.skip("needs a GPU", allow_module_level=True)

from combine_ep_layout_amd import binding as B  # noqa: E402
from tests import router_ref as R  # noqa: E402

DEV = "cuda:0"


def test_a_workspace_for_the_largest_batch_serves_the_smaller_ones():
    most = [(33000, 8), (33000, 300)]  # tokens, experts
    for (T, E), smaller in zip(most, ([33000, 32768, 24577, 24576, 12289, 12288, 700, 1], [33000, 32769, 32768, 16385, 16384, 1])):
        wsb = B.ep_router_workspace_bytes(T, E, 1)
        ws = torch.full((wsb + 64,), 0xA5, dtype=torch.uint8, device=DEV)
        l = torch.randn(T, E, generator=torch.Generator(device=DEV).manual_seed(E), device=DEV)
        for n in smaller:
            print(f"[workspace] T={n} E={E} of {T}", flush=True)
            idx, w = torch.empty(n, 2, dtype=torch.int32, device=DEV), torch.empty(n, 2, device=DEV)
            counts, tokens = torch.empty(1, E, dtype=torch.int32, device=DEV), torch.empty(3, dtype=torch.int32, device=DEV)
            losses = torch.empty(2, device=DEV)
            B.ep_router(l, None, None, None, n, E, 2, 1, B.EP_FP32, B.EP_SOFTMAX, 1, 1.0, 0, idx, w, counts, tokens, losses, losses[1:],
                        ws, wsb)
            torch.cuda.synchronize()
            ids = R.choose(l[:n].double(), 2, "softmax")
            want, number, (balance, db), (z, dz) = R.statistics(l[:n].double(), ids, "softmax", None)
            assert torch.equal(idx.long(), ids) and torch.equal(counts.long(), want) and torch.equal(tokens.long(), number)
            assert abs(float(losses[0]) - balance) <= db + R.U * balance and abs(float(losses[1]) - z) <= dz + R.U * z
            assert bool((ws[wsb:] == 0xA5).all())
