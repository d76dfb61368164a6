"""Products on buffers that are mostly padding: few experts with rows among many, wide alignment.

How many experts have rows is found on the device, and with it how the work is shared out; the results
have to be right on every side of that choice, under caps, and whatever the padding holds.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - only on CPU hosts
    pytest.skip("needs a GPU", allow_module_level=True)

from combine_ep_layout_amd import binding as B  # noqa: E402
from tests import experts_ref as R  # noqa: E402

DEV = "cuda:0"
KIND = {"bf16": B.EP_BF16, "fp8": B.EP_FP8_E4M3, "fp4": B.EP_FP4X2}

CASES = [
    # kind, E, K, N, {expert: rows}, A
    ("bf16", 64, 264, 1024, {0: 1}, 16),
    ("bf16", 64, 136, 904, {63: 17, 5: 1}, 128),
    ("fp8", 256, 384, 1024, {3: 4, 100: 1, 255: 33}, 16),
    ("fp4", 256, 640, 520, {7: 1, 8: 16}, 64),
    ("fp4", 100, 128, 1032, {i: 1 + i % 3 for i in range(0, 96, 8)}, 16),  # 12 experts of 9 tiles: enough
    ("bf16", 100, 128, 1032, {i: 20 for i in range(0, 56, 8)}, 32),  # 7 of 9 tiles, 20 rows each
    ("bf16", 100, 128, 1032, {i: 16 for i in range(0, 56, 8)}, 32),  # the same with 16 rows
    ("fp8", 1024, 128, 200, {255: 2, 256: 3, 600: 18, 1023: 1}, 8),  # counts behind the first 256
    ("bf16", 1024, 64, 128, {i: 1 for i in range(0, 1024, 10)}, 4),  # 103 experts of one tile
    ("fp8", 64, 1152, 1024, {i: 0 for i in range(64)}, 16),  # no rows at all
]


def _weights(E, N, K, kind, gen):
    if kind == "bf16":
        return torch.randn(E, N, K, generator=gen, device=DEV).mul_(K ** -0.5).bfloat16(), None
    scales = (torch.rand(E, N, K // 128, generator=gen, device=DEV) + 0.3) * K ** -0.5
    if kind == "fp8":
        return torch.randn(E, N, K, generator=gen, device=DEV).to(torch.float8_e4m3fn).view(torch.uint8), scales
    return torch.randint(0, 256, (E, N, K // 2), generator=gen, device=DEV, dtype=torch.uint8), scales


@pytest.mark.parametrize("out", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind,E,K,N,have,A", CASES)
def test_matvec(kind, E, K, N, have, A, out):
    print(f"[padded] {kind} E={E} K={K} N={N} {have} A={A} {out}", flush=True)
    gen = torch.Generator(device=DEV).manual_seed(E + N)
    counts = [have.get(e, 0) for e in range(E)]
    off = [0]
    for n in counts:
        off.append(off[-1] + -(-n // A) * A)
    cap = sum(counts) + E * (A - 1)  # as a caller sizes it before it knows the routing
    i32 = dict(dtype=torch.int32, device=DEV)
    c, o = torch.tensor(counts, **i32), torch.tensor(off, **i32)
    w, s = _weights(E, N, K, kind, gen)
    live = torch.zeros(cap, dtype=torch.bool, device=DEV)
    for e, n in enumerate(counts):
        live[off[e]:off[e] + n] = True
    x = torch.full((cap, K), float("nan"), dtype=torch.bfloat16, device=DEV)
    x[live] = torch.randn(int(live.sum()), K, generator=gen, device=DEV).bfloat16()
    dt = B.EP_FP32 if out is torch.float32 else B.EP_BF16
    results = []
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    for limit in (0, 1, 6):
        y = torch.full((cap, N), -7.0, dtype=out, device=DEV)
        torch.cuda.synchronize()
        B.ep_set_workgroup_limit(st, limit)
        try:
            B.ep_expert_matvec(x, w, s, c, o, E, cap, K, N, KIND[kind], y, dt, st)
            st.synchronize()
        finally:
            B.ep_set_workgroup_limit(st, 0)
        results.append(y)
    y = results[0]
    assert all(torch.equal(y, r) for r in results[1:])
    assert bool((y[~live] == -7.0).all())
    for e, n in enumerate(counts):
        if n:
            z = x[off[e]:off[e] + n].double()
            want, err = R.product(z, torch.zeros_like(z), R.values(w[e], None if s is None else s[e], kind))
            R.near(y[off[e]:off[e] + n], want, err, out)
