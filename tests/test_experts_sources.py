"""What the kernels' signatures promise the compiler against what the header allows its callers.

A pointer that is __restrict__ promises that nothing it reads is written through another one. Where the
header lets an input be an output ("may be"), neither side may carry that promise: the compiler would be
free to store the output before it has loaded the input of the same element.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_ep_layout_amd", "csrc")
IN_PLACE = [("ep_swiglu.hip", "ep_swiglu_backward_rows", "dh", "h"), ("ep_expert.hip", "ep_moe_down", "bias", "out"),
            ("ep_wgrad.hip", "ep_expert_wgrad_tiles", "previous", "dw")]


def _parameters(source, kernel):
    text = re.sub(r"//[^\n]*", "", source)
    found = re.search(r"\b" + kernel + r"\s*\(([^)]*)\)", text)
    assert found, kernel
    return {p.split()[-1].lstrip("*"): p for p in found.group(1).split(",")}


@pytest.mark.parametrize("source,kernel,read,written", IN_PLACE)
def test_operands_that_may_be_one_make_no_promise(source, kernel, read, written):
    with open(os.path.join(CSRC, source)) as f:
        params = _parameters(f.read(), kernel)
    assert "__restrict__" not in params[read] and "__restrict__" not in params[written]
