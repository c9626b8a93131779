"""Waits that one lane makes for its warp, read from the kernels' sources (no GPU
needed): the other lanes are ordered behind that lane by a barrier of the warp, and
by nothing less (a shuffle or a vote orders no memory), before they read what was
waited for."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "contextual_sparsity_decode_gb300", "csrc")
ONE_LANE = re.compile(r"if \(lane == 0 && !(?:tc::)?mbar_wait\w*\(")


def _after_statement(text, at):
    """The code behind the `if` that begins at `at`, without comments."""
    depth, i = 0, text.index("(", at)
    while True:                                   # its condition
        depth += {"(": 1, ")": -1}.get(text[i], 0)
        i += 1
        if depth == 0:
            break
    rest = text[i:]
    if not rest.lstrip().startswith("{"):
        return rest[rest.index(";") + 1:].lstrip()
    depth, j = 0, rest.index("{")
    while True:                                   # its block
        depth += {"{": 1, "}": -1}.get(rest[j], 0)
        j += 1
        if depth == 0:
            return rest[j:].lstrip()


def _waits():
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu*"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for m in ONE_LANE.finditer(text):
            yield os.path.basename(path), text, m.start()


@pytest.mark.parametrize("name", ["k_beam.cu", "k_sample.cu"])
def test_a_lane_that_waits_for_its_warp_is_followed_by_a_warp_barrier(name):
    found = [(text, at) for file, text, at in _waits() if file == name]
    assert found
    for text, at in found:
        assert _after_statement(text, at).startswith("__syncwarp();")


def test_no_other_kernel_waits_by_one_lane():
    assert {file for file, _, _ in _waits()} == {"k_beam.cu", "k_sample.cu"}
