"""ep_router_workspace_bytes never falls where a call grows: a buffer for the largest call serves every smaller one."""
import os
import random

import pytest

from combine_ep_layout_amd import binding as B


@pytest.fixture(scope="module", autouse=True)
def L():
    if not os.path.exists(B.LIB_PATH):
        from combine_ep_layout_amd import build
        build.build()
    return B.lib()


size = B.ep_router_workspace_bytes


@pytest.mark.parametrize("E,S", [(1, 1), (60, 1), (256, 1), (256, 37), (257, 1), (1024, 1), (1024, 5000)])
def test_more_tokens_never_need_less(E, S):
    # tokens around multiples of 16 tokens for every workgroup that runs at once, three or four a compute unit
    tokens = sorted({n * 16 * w * 256 + d for w in (3, 4) for n in range(1, 18) for d in (-1, 0, 1)} | set(range(0, 700, 7)))
    sizes = [size(T, E, S) for T in tokens]
    assert all(a <= b for a, b in zip(sizes, sizes[1:])), [(T, a, b) for T, a, b in zip(tokens, sizes, sizes[1:]) if a > b][:3]


@pytest.mark.parametrize("T", [0, 1, 4096, 12289, 16385, 100000, 300000, 1 << 24, 2 ** 31 - 4097])
def test_more_experts_never_need_less(T):
    for S in (1, 9, 300, 40000):
        sizes = [size(T, E, S) for E in range(1, 1025)]
        assert all(a <= b for a, b in zip(sizes, sizes[1:])), (S, [E for E, (a, b) in enumerate(zip(sizes, sizes[1:]), 1) if a > b])


@pytest.mark.parametrize("T,E", [(0, 16), (4096, 256), (100000, 1024), (1 << 22, 8), (1 << 28, 256), (2 ** 31 - 4097, 1024)])
def test_more_sequences_never_need_less(T, E):
    sizes = [size(T, E, S) for S in range(1, B.EP_MAX_SEQUENCES + 1, 13)]
    assert all(a <= b for a, b in zip(sizes, sizes[1:]))


def test_drawn_calls():
    rng = random.Random(4)
    for _ in range(20000):
        T, E, S = rng.randrange(1 << rng.randrange(1, 31)), rng.randrange(1, 1025), rng.randrange(1, 1 << rng.randrange(1, 17))
        more = T + rng.randrange(1 << rng.randrange(1, 20)), min(1024, E + rng.randrange(40)), min(65536, S + rng.randrange(40))
        assert 0 < size(T, E, S) <= size(*more), (T, E, S, more)
