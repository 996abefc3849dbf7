"""Rules that the scan's and the norms' sources keep, read from the text (no GPU).

A read-only load (__ldg) is allowed of what nothing writes while the kernel is resident:
the compiler may move it over a wait for the kernel before, and the read-only path may
answer from an older line.  So not of the workspace, whose writers may still run when the
reader's blocks start, and not of an array that the call may write in place.
"""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ssm_decode_02_b200", "csrc")
FILES = sorted(f for f in os.listdir(CSRC) if f.startswith(("scan", "norm", "tc.")))


def text(name):
    with open(os.path.join(CSRC, name)) as f:
        return f.read()


def arguments(source, call):
    """The argument of every `call(` in the source, to its closing parenthesis."""
    for m in re.finditer(re.escape(call) + r"\(", source):
        depth, at = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(source[at], 0)
            at += 1
        yield source[m.end():at - 1]


@pytest.mark.parametrize("name", [f for f in FILES if f.startswith("scan")])
def test_read_only_loads_of_the_scan_are_of_its_inputs(name):
    for arg in arguments(text(name), "__ldg"):
        assert re.search(r"\bp\.(x|dt|A|D|decay|cu)\b", arg), (name, arg)


def test_read_only_loads_of_the_norms_are_of_their_inputs():
    """Through one function, asked for by the loads of arrays that no call writes: not the partial
    sums, not the residual (h may be written over it) and not dh (dresidual may be)."""
    source = text("norm.cu")
    for arg in arguments(source, "__ldg"):
        assert re.search(r"(>\(p\)|^p)( \+ 1)?$", arg), arg                # of load_fixed
    assert set(re.findall(r"(\w+)\(const \w+\* p\) \{[^}]*__ldg", source)) == {"load_fixed"}
    fetches = {(m, a.rsplit(",", 1)[1].strip()) for m in ("xs", "ys", "ss", "hs") for a in arguments(source, m + ".fetch")}
    assert fetches == {("xs", "true"), ("ys", "true"), ("hs", "false"), ("ss", "MODE != kResidual"), ("ss", "true")}
