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


def _asm(code):
    """The instructions of every asm statement."""
    for m in re.finditer(r'asm(?:\s+volatile)?\s*\(((?:\s*"(?:[^"\\]|\\.)*")+)', code):
        yield re.sub(r'"\s*"', "", m.group(1)).strip().strip('"')


def test_arrivals_at_another_cta_release_to_the_cluster():
    """What one CTA's threads wrote is another CTA's thread's to see only behind a release at cluster scope (the form
    without a scope is of the CTA's).  Without release: TMEM columns that have been read, which hand over no memory."""
    remote = []
    for name in sorted(os.listdir(CSRC)):
        code = _code(name)
        remote += [(name, i) for text in _asm(code) for i in re.findall(r"mbarrier\.arrive[\w.:]*", text)
                   if "shared::cluster" in i and "commit" not in text]
        for call in re.findall(r"mbar_arrive_remote_relaxed\(\s*(\w+)\(\s*(\w+)", code):
            assert call in (("map_to_rank", "tempty_bar"),), (name, call)
    assert {i for _, i in remote} == {"mbarrier.arrive.release.cluster.shared::cluster.b64",
                                      "mbarrier.arrive.relaxed.cluster.shared::cluster.b64"}, remote


def test_threads_waiting_for_another_cta_acquire_from_the_cluster():
    """A barrier that the other CTA of a pair arrives on (mbar_arrive_remote) is waited for with acquire at cluster scope."""
    for name in sorted(f for f in os.listdir(CSRC) if f.endswith(".cu")):
        code = _code(name)
        for bar in set(re.findall(r"mbar_arrive_remote(?:_relaxed)?\(\s*map_to_rank\(\s*(\w+)\(", code)):
            waits = re.findall(r"(\w+)\(\s*" + bar + r"\(", code)
            waits = [w for w in waits if "wait" in w]
            assert waits and all("cluster" in w for w in waits), (name, bar, waits)
