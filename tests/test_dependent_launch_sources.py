"""Source check: kernels that run as programmatic dependent launches read global memory coherently.

Such a kernel's lifetime begins while the kernel before it still runs, so nothing that one may write is
read-only for that lifetime, which is what the non-coherent loads (ld.global.nc, __ldg) require."""
import os
import re

import pytest

from conftest import ROOT

CSRC = os.path.join(ROOT, "transformer_ffn_block_gb300", "csrc")
NON_COHERENT = re.compile(r"\b(ld16_ro|ld16_ro_stream|__ldg|__ldcs_nc)\s*\(|ld\.global[.\w:]*\.nc\b|\b__restrict__\b")


def _code(path):
    """The source without comments."""
    text = open(path).read()
    text = re.sub(r"/\*.*?\*/", " ", text, flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


def _functions(code):
    """(head, body) of every brace block at namespace level that follows a parameter list."""
    i = 0
    while (m := re.compile(r"\)\s*\{").search(code, i)) is not None:
        depth, j = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(code[j], 0)
            j += 1
        head = code[max(code.rfind("}", 0, m.start()), code.rfind(";", 0, m.start())) + 1:m.start()]
        yield head, code[m.end():j]
        i = j


SOURCES = sorted(f for f in os.listdir(CSRC) if f.endswith(".cu"))


def test_there_are_dependent_kernels():
    waiting = [f for f in SOURCES if "pdl_wait();" in _code(os.path.join(CSRC, f))]
    assert {"decode.cu", "elementwise.cu", "gemm_fp8.cu", "norm.cu", "linear.cu", "few_rows.cu", "skinny.cu"} <= set(waiting)


@pytest.mark.parametrize("name", SOURCES)
def test_dependent_kernels_load_coherently(name):
    """In a file with such kernels the non-coherent loads stay within kernels that are launched plainly."""
    code = _code(os.path.join(CSRC, name))
    if "pdl_wait();" not in code:
        return
    for head, body in _functions(code):
        plain_kernel = "__global__" in head and "pdl_wait();" not in body
        found = NON_COHERENT.search(head + body)
        assert plain_kernel or found is None, (name, re.findall(r"(\w+)\s*\(", head)[-1], found.group(0))


@pytest.mark.parametrize("name", SOURCES)
def test_settled_loads_follow_the_wait(name):
    """ld16_settled reads through a pointer that behind_wait() gives, after the kernel's pdl_wait()."""
    for head, body in _functions(_code(os.path.join(CSRC, name))):
        given = {}
        for m in re.finditer(r"(\w+) = behind_wait\(", body):
            given[m.group(1)] = m.start()
            assert 0 <= body.find("pdl_wait();") < m.start(), (name, m.group(1))
        for m in re.finditer(r"ld16_settled\((\w+)", body):
            assert m.group(1) in given and given[m.group(1)] < m.start(), (name, m.group(0))


def test_inline_loads_keep_their_order():
    """A load written as asm may move across the wait unless it is volatile and clobbers memory
    (ld16_settled: see above)."""
    for f in sorted(os.listdir(CSRC)):
        code = re.sub(r"uint4 ld16_settled\(.*?\n}", "", _code(os.path.join(CSRC, f)), flags=re.S)
        for m in re.finditer(r"asm(\s+volatile)?\s*\(([^;]*?ld\.(?:global|shared)[^;]*?;[^;]*?)\);", code, flags=re.S):
            assert m.group(1) and '"memory"' in m.group(2), (f, " ".join(m.group(0).split())[:120])
