"""Where a tensor-core role gives up (csrc), read from the sources, without a GPU: it commits its
MMAs to a barrier of its own and waits for that, so that none is in flight when the block goes on.
A barrier that two roles share completes for one by the other's commit, and twice is as if never."""
import re

import pytest

from test_dependent_launch_cpu import code

# kernels whose blocks multiply by more than one warp, and the index of such a warp
TWO = [("f8_mm.cu", "k_f8_wide", "h")]
ONE = [("f8_mm.cu", "k_f8_mm"), ("mx_mm.cu", "k_mx_mm"), ("grad_w.cu", "k_grad_w")]
COMMIT = re.compile(r"(?:umma_commit|pair_commit|wide_commit<\w+>)\s*\(\s*&drain((?:\[\w+\])?)")
WAIT = re.compile(r"mbar_wait_for\s*\(\s*&drain((?:\[\w+\])?)")
INIT = re.compile(r"mbar_init\s*\(\s*&drain((?:\[\w+\])?)")


def body(name, kernel):
    text = code(name)
    start = re.search(r"\b%s\((?=const)" % kernel, text).start()
    depth, end = 0, text.index("{", text.index(")", start))
    for end in range(end, len(text)):
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        if depth == 0:
            break
    return text[start:end]


@pytest.mark.parametrize("name,kernel,index", TWO)
def test_each_multiplying_warp_has_its_own_barrier(name, kernel, index):
    text = body(name, kernel)
    assert re.search(r"uint64_t[^;]*\bdrain\[2\]", text)
    own = "[%s]" % index
    assert COMMIT.findall(text) == [own] and WAIT.findall(text) == [own]
    assert sorted(INIT.findall(text)) in (["[0]", "[1]"], ["[i]"])


@pytest.mark.parametrize("name,kernel", ONE)
def test_one_multiplying_warp_has_one_barrier(name, kernel):
    text = body(name, kernel)
    assert COMMIT.findall(text) == [""] and WAIT.findall(text) == [""] and INIT.findall(text) == [""]
