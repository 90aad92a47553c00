"""Source checks of how the warps and CTAs of a kernel wait for one another, where a wrong wait shows in few runs or none."""
import os
import re

from conftest import ROOT

CSRC = os.path.join(ROOT, "transformer_ffn_block_gb300", "csrc")


def _code(name):
    """The source without comments."""
    text = re.sub(r"/\*.*?\*/", " ", open(os.path.join(CSRC, name)).read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


def test_the_table_is_awaited_by_its_one_phase():
    """The barrier of the groups' table has one arrival in a launch, which completes the phase of parity 0.  A wait for
    the other parity returns only while that arrival is still to come, and never behind it."""
    code = _code("grouped.cu")
    assert len(re.findall(r"mbar_arrive\w*\(\s*table_bar", code)) == 1
    waits = re.findall(r"\w*wait\w*\(\s*table_bar\s*,\s*([^;{]*?),\s*abort_flag", code)
    assert waits and all(re.fullmatch(r"0u?", w.strip()) for w in waits), waits
