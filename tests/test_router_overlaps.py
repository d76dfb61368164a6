"""Outputs of the router's operators that share memory with another operand are refused on the host."""
import itertools
import os

import pytest

from combine_ep_layout_amd import binding as B

MB = 1 << 20
NAMES = ["l", "bias", "mask", "seq", "idx", "w", "c", "n", "b", "z", "ws", "dw", "db", "dz", "d"]
PLACE = {name: (n + 1) * 16 * MB for n, name in enumerate(NAMES)}  # never dereferenced
T, E, K, S = 50, 16, 2, 3
BYTES = dict(l=T * E * 4, bias=E * 4, mask=T, seq=(S + 1) * 4, idx=T * K * 4, w=T * K * 4, c=S * E * 4, n=(S + 2) * 4, b=4, z=4,
             dw=T * K * 4, db=4, dz=4, d=T * E * 4)


@pytest.fixture(scope="module", autouse=True)
def L():
    if not os.path.exists(B.LIB_PATH):
        from combine_ep_layout_amd import build
        build.build()
    BYTES["ws"] = B.ep_router_workspace_bytes(T, E, S)
    return B.lib()


def _refused(fn, args):
    with pytest.raises(B.EpError) as ei:
        fn(*args)
    said = B.ep_last_error()
    return ei.value.code == B.EP_EINVAL and said.startswith(fn.__name__ + ":") and "overlap" in said


def router(given=0, **at):
    p = {**PLACE, **at}
    return (p["l"], None if given else p["bias"], None if given else p["mask"], p["seq"], T, E, K, S, B.EP_FP32, B.EP_SOFTMAX, 1, 1.0,
            given, p["idx"], p["w"], p["c"], p["n"], p["b"], p["z"], p["ws"], BYTES["ws"])


def backward(**at):
    p = {**PLACE, **at}
    return p["l"], p["idx"], p["seq"], p["c"], p["n"], p["dw"], p["db"], p["dz"], T, E, K, S, B.EP_FP32, B.EP_SOFTMAX, 1, 1.0, p["d"]


OUT = ["idx", "w", "c", "n", "b", "z", "ws"]


def _ends(out, other):
    """Places of `out` that reach just into `other`, aligned as both want it."""
    step = 16 if out in ("ws", "d") else 4
    last = (BYTES[other] - 1) // step * step
    return {PLACE[other], PLACE[other] + last, PLACE[other] - (BYTES[out] - 1) // step * step}


@pytest.mark.parametrize("out,other", [(a, b) for a, b in itertools.product(OUT, ["l", "bias", "mask", "seq"] + OUT) if a != b])
def test_router_results_over_an_operand(out, other):
    for at in _ends(out, other):
        assert _refused(B.ep_router, router(**{out: at})), at


@pytest.mark.parametrize("out", [n for n in OUT if n != "idx"])
def test_router_results_over_given_ids(out):
    for at in _ends(out, "idx"):
        assert _refused(B.ep_router, router(given=1, **{out: at})), at


@pytest.mark.parametrize("other", ["l", "idx", "seq", "c", "n", "dw", "db", "dz"])
def test_a_gradient_over_an_operand(other):
    for at in _ends("d", other):
        assert _refused(B.ep_router_backward, backward(d=at)), at


def test_operands_beside_each_other_are_not_refused():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a call that is not refused would run on addresses that do not exist")
    at, row = MB, {}
    for name in NAMES:  # one behind the other
        row[name] = at = (at + 15) // 16 * 16
        at += BYTES[name]
    assert not _refused(B.ep_router, router(**row)) and not _refused(B.ep_router_backward, backward(**row))
    assert not _refused(B.ep_router, router(given=1, **row))
    # losses and gradients of one array each, as a program keeps them; what is only read may overlap
    one = dict(b=MB, z=MB + 4, db=2 * MB, dz=2 * MB + 4)
    assert not _refused(B.ep_router, router(**one)) and not _refused(B.ep_router_backward, backward(**one))
    assert not _refused(B.ep_router_backward, backward(db=PLACE["dw"], dz=PLACE["dw"]))
