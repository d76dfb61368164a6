"""Outputs of the 8-bit integer operators that share memory with another operand are refused on the host."""
import os

import pytest

from combine_ep_layout_amd import binding as B

MB = 1 << 20
PLACE = {name: (n + 1) * 16 * MB for n, name in enumerate(["x", "s", "w", "ws", "c", "o", "y", "codes"])}  # never dereferenced


@pytest.fixture(scope="module", autouse=True)
def L():
    if not os.path.exists(B.LIB_PATH):
        from combine_ep_layout_amd import build
        build.build()
    return B.lib()


def _refused(fn, args):
    with pytest.raises(B.EpError) as ei:
        fn(*args)
    said = B.ep_last_error()
    return ei.value.code == B.EP_EINVAL and said.startswith(fn.__name__ + ":") and "overlap" in said


def _no_gpu():
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("a call that is not refused would run on addresses that do not exist")


E, CAP, K, N, COLS = 4, 64, 512, 256, 3


def matmul(**at):
    p = {**PLACE, **at}
    return p["x"], p["s"], COLS, p["w"], p["ws"], p["c"], p["o"], E, CAP, K, N, p["y"], B.EP_FP32


BYTES = dict(x=CAP * K, s=((CAP - 1) * COLS + 1) * 4, w=E * N * K, ws=E * N * 4, c=E * 4, o=E * 4)


@pytest.mark.parametrize("name", BYTES)
def test_matmul_results_over_an_operand(name):
    size = CAP * N * 4
    for at in (0, BYTES[name] - 4, 16 - size, 16):
        at = at // 16 * 16  # rows need 16 bytes
        if -size < at < BYTES[name]:
            assert _refused(B.ep_quantized_matmul, matmul(y=PLACE[name] + at)), at


@pytest.mark.parametrize("name", BYTES)
def test_matmul_results_beside_an_operand_are_not_refused(name):
    _no_gpu()
    for y in (PLACE[name] + (BYTES[name] + 15) // 16 * 16, PLACE[name] - CAP * N * 4):
        assert not _refused(B.ep_quantized_matmul, matmul(y=y))


def quantize(**at):
    p = {**PLACE, **at}
    return p["x"], p["c"], p["o"], E, CAP, K, B.EP_FP32, p["codes"], p["s"], COLS


@pytest.mark.parametrize("fn,factor", [(B.ep_quantize_rows, 1), (B.ep_swiglu_quantize, 2)], ids=["rows", "gated"])
@pytest.mark.parametrize("name", ["x", "codes", "c", "o"])
def test_scales_over_an_operand(fn, factor, name):
    size = {"x": CAP * K * 4 * factor, "codes": CAP * K, "c": E * 4, "o": E * 4}[name]
    for at in (0, size - 4, 4 - CAP * COLS * 4):
        assert _refused(fn, quantize(s=PLACE[name] + at)), at
    if name != "codes":
        for at in (0, size - 4, 16 - CAP * K):
            assert _refused(fn, quantize(codes=PLACE[name] + at // 16 * 16)), at


@pytest.mark.parametrize("fn,factor", [(B.ep_quantize_rows, 1), (B.ep_swiglu_quantize, 2)], ids=["rows", "gated"])
def test_scales_beside_an_operand_are_not_refused(fn, factor):
    _no_gpu()
    for s in (PLACE["x"] + CAP * K * 4 * factor, PLACE["codes"] + CAP * K, PLACE["codes"] - CAP * COLS * 4, PLACE["c"] + 4 * E):
        assert not _refused(fn, quantize(s=s))
