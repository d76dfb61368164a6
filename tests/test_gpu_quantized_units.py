"""Units of few rows that are shared out between the two launches of ep_quantized_matmul.

When there are fewer tiles than workgroups, the others take the first `early` units of the experts with few rows, and
the second launch begins behind those. Every case here has 0 < early < units, by a copy of the kernels' rule, so that a
unit left out or taken twice at the border shows. Results are determined to the last bit.
"""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - only on CPU hosts
    pytest.skip("needs a GPU", allow_module_level=True)

from combine_ep_layout_amd import binding as B  # noqa: E402
from tests.test_gpu_quantized import DEV, TYPE, _codes, _exact, _gen, _matmul, _spans  # noqa: E402

FEW, SIDE, BESIDE, XCDS = 32, 256, 6, 8


def plan(counts, N, grid):
    """(tiles, units, early, wide, the most rows of an expert with few, XCDs with more tiles than workgroups)"""
    up = lambda n, d: -(-n // d)  # noqa: E731
    tiles = sum(up(n, SIDE) * up(N, SIDE) for n in counts if n > FEW)
    few = [n for n in counts if 0 < n <= FEW]
    wide = len(few) * up(N, 64) >= grid
    units = len(few) * up(N, 64 if wide else 16)
    idle = grid - tiles if 0 < tiles < grid else 0
    early = min(idle * BESIDE * (1 if wide else 4), units)
    active = min(grid, XCDS)
    share = [tiles * (x + 1) // active - tiles * x // active for x in range(active)]
    have = [up(grid - x, XCDS) for x in range(active)]
    return tiles, units, early, wide, max(few, default=0), sum(s > h for s, h in zip(share, have))


def some(most, n, seed):
    g = torch.Generator().manual_seed(seed)
    got = torch.randint(0, most + 1, (n,), generator=g).tolist()
    got[n // 2] = most
    return got


CASES = [
    # K, N, counts, workgroups, wide, rows above 16, XCDs with more tiles than workgroups
    (256, 4096, [300, *some(16, 30, 1), 40, *some(16, 31, 2), 60], 256, True, False, False),
    (144, 4096, [*some(32, 61, 3), 33, 257, 64], 256, True, True, False),
    (256, 4096, [*some(16, 40, 4), 3000], 256, True, False, False),
    (512, 2056, [70, *some(32, 100, 5)], 256, True, True, False),
    (64, 256, [2800, *some(16, 62, 6)] + [2800] * 19, 256, False, False, False),
    (64, 264, [1400, *some(32, 50, 7)] + [1400] * 18, 256, False, True, False),
    (128, 256, [300, 9, 700, 600, 40, 3, 50, 60], 12, False, False, True),
    (128, 256, [300, 32, 700, 600, 40, 17, 50, 60], 12, False, True, True),
    (272, 1024, [33, 100, *some(16, 9, 8), 256], 13, True, False, True),
    (80, 512, [40, *some(32, 12, 9)], 3, True, True, False),
    (80, 776, [200, *some(32, 62, 10)], 100, True, True, False),
]


@pytest.mark.parametrize("K,N,counts,grid,wide,tall,crowded", CASES)
def test_units_on_both_sides_of_the_border(K, N, counts, grid, wide, tall, crowded):
    tiles, units, early, is_wide, most, over = plan(counts, N, grid)
    print(f"[units] K={K} N={N} experts={len(counts)} workgroups={grid}: {tiles} tiles, {early} of {units} units beside them", flush=True)
    assert 0 < early < units and is_wide == wide and (most > 16) == tall and (over > 0) == crowded
    gen = _gen(41, K, N, len(counts))
    E = len(counts)
    c, o, rows, real, cap = _spans(counts, 8, 3)
    x, w = _codes((cap, K), gen), _codes((E, N, K), gen)
    sx, sw = torch.rand(cap, 1, generator=gen, device=DEV) + 0.1, torch.randn(E, N, generator=gen, device=DEV)
    s = torch.cuda.Stream()
    for out in ("bf16", "fp32"):
        y = torch.full((cap, N), -7.0, dtype=TYPE[out], device=DEV)
        torch.cuda.synchronize()
        if grid < 256:
            B.ep_set_workgroup_limit(s, grid)
        try:
            _matmul(x, sx, w, sw, c, o, E, cap, y, s)
            torch.cuda.synchronize()
        finally:
            if grid < 256:
                B.ep_set_workgroup_limit(s, 0)
        wrong = [e for e, r in enumerate(rows) if len(r) and not torch.equal(
            y[r.start:r.stop], _exact(x[r.start:r.stop], sx[r.start:r.stop, 0], w[e], sw[e], TYPE[out]))]
        assert not wrong, f"experts {wrong}"
        assert bool((y[~real] == -7.0).all())
