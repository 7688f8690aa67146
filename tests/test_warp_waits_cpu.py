"""Waits that a warp shares out among its lanes (csrc/*.cu, *.cuh), read from the sources, without a
GPU: a lane that polls one barrier has acquired that one alone, and a vote orders no memory between
lanes, so a vote over different barriers is followed by __syncwarp before anything is read."""
import glob
import os
import re

import pytest

from test_dependent_launch_cpu import CSRC, code

SOURCES = sorted(os.path.basename(p) for e in ("*.cu", "*.cuh") for p in glob.glob(os.path.join(CSRC, e)))
VOTE = re.compile(r"__(?:all|any)_sync\s*\(")


def statement(text, start):
    """From `start` to the semicolon that ends it, and the statement behind that one."""
    end = text.index(";", start)
    return text[start:end], text[end + 1:text.index(";", end + 1)].strip()


def unordered(text):
    """Votes over waits whose barrier depends on the lane, with no __syncwarp behind them."""
    bad = []
    for m in VOTE.finditer(text):
        vote, behind = statement(text, m.start())
        wait = re.search(r"mbar_(?:wait|wait_for|ready)\s*\(\s*([^,]*)", vote)
        if wait and "?" in wait.group(1) and not behind.startswith("__syncwarp("):
            bad.append(vote)
    return bad


@pytest.mark.parametrize("name", SOURCES)
def test_a_vote_over_two_barriers_is_ordered(name):
    assert not unordered(code(name))


def test_the_check_sees_each_form():
    vote = "ok = __all_sync(~0u, mbar_wait_for(lane == 0 ? &a : &b, lane == 0 ? p : q, n));"
    assert unordered(vote + " if (!ok) break;") and unordered(vote + " tc_fence_after();")
    assert not unordered(vote + " __syncwarp(); return ok;")
    assert not unordered("ok = __all_sync(~0u, mbar_wait_for(&a[i], i ? 1u : 0u, n)); if (!ok) break;")
