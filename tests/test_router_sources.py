"""Where lanes of one wave exchange values through LDS in the router's kernels: what one lane writes and another reads
or writes has to be ordered by a fence, because the compiler only sees one lane's addresses."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_ep_layout_amd", "csrc")


def test_the_gradients_exchange_is_fenced():
    with open(os.path.join(CSRC, "ep_router.hip")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    # a lane's columns cleared, entries added by their lanes, columns read, entries cleared again
    steps = ["mine[column<L, V>(i, j)] = 0.f;", "mine[ids[0]] = sum;", "out[j] = mine[column<L, V>(i, j)];",
             "if (ids[b] >= 0) mine[ids[b]] = 0.f;", "if (!there) continue;"]
    at = [text.index(s) for s in steps]
    assert at == sorted(at)
    for a, b in zip(at, at[1:]):
        assert "__builtin_amdgcn_fence(" in text[a:b], text[a:b]
