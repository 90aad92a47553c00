"""The Python binding's own host code: what needs no GPU."""
import subprocess
import sys
import threading
import time

import pytest
import torch

from conftest import ROOT

from test_abi import A, lib  # noqa: F401  (lib: the module's build-and-load fixture)


@pytest.fixture
def fresh(lib, monkeypatch):  # noqa: F811
    """The binding as before its first call."""
    for name in ("_torch", "_get_device", "_get_stream"):
        monkeypatch.setattr(lib, name, None)
    return lib


def test_first_calls_from_many_threads(fresh, monkeypatch):
    """While one thread looks the device up for the first time, the others wait for it."""
    def slow():
        time.sleep(0.1)
        return True

    monkeypatch.setattr(torch.cuda, "is_available", slow)
    monkeypatch.setattr(torch.cuda, "init", lambda: time.sleep(0.05))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 3, raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda d: 1000 + d, raising=False)
    start, seen = threading.Barrier(8), []

    def call(i):
        start.wait()
        time.sleep(0.02 * i)
        seen.append(fresh._current_device() if i % 2 else fresh._stream(None) - 1000)

    threads = [threading.Thread(target=call, args=(i,)) for i in range(8)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert seen == [3] * 8


RAW = """
import sys
import transformer_ffn_block_gb300 as q
A = 4096
for call in (lambda: q.qffn_linear(A, None, A, A, None, None, 9, 4, 32, 64, A, 4096, stream=0),
             lambda: q.qffn_gated_linear(A, A, A, 9, 4, 32, 64, A, 4096, stream=0),
             lambda: q.qffn_layernorm_absmax(None, A, A, A, None, None, A, A, None, -1.0, 4, 64, stream=0),
             lambda: q.qffn_rmsnorm_backward(A, A, None, A, None, A, A, A, -4, 64, False, A, 4096, stream=0)):
    try:
        call()
    except q.QffnError as e:
        assert e.status == 1
    else:
        raise SystemExit("not refused")
assert "torch" not in sys.modules, "torch was imported"
"""


def test_raw_addresses_need_no_torch(lib):  # noqa: F811
    """Calls with bare addresses and a stream reach the library without importing torch."""
    r = subprocess.run([sys.executable, "-c", RAW], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
