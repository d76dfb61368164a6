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


# Where the lanes of one wave exchange values through LDS without a barrier of the workgroup: what one lane
# writes and another reads has to be ordered by a fence, because the compiler only sees one lane's addresses.
EXCHANGES = [("ep_wgrad.hip", "*(f32x4 *)(mine +", "const char *from = mine +", "raw_buffer_store_b128(w, to"),
             ("ep_expert.hip", "*(u32x4 *)(slot +", "*(const u32x4 *)(slot +", "return got")]


@pytest.mark.parametrize("source,write,read,after", EXCHANGES)
def test_values_that_change_lanes_are_fenced(source, write, read, after):
    with open(os.path.join(CSRC, source)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    at = text.index(write)
    then = text.index(read, at + len(write))
    assert "__builtin_amdgcn_fence(" in text[at:then], "before the read"
    end = text.index(after, then)
    # up to the end of the loop body or function that writes the place again
    assert "__builtin_amdgcn_fence(" in text[then:end + 200], "before the next write"
