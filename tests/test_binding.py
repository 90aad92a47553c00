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


class _Reached:
    """In place of the C library: every call succeeds and is counted."""

    def __init__(self):
        self.calls = 0

    def __getattr__(self, name):
        def call(*args):
            self.calls += 1
            return 0
        return call


@pytest.fixture
def on_cpu(lib, monkeypatch):  # noqa: F811
    """The binding with CPU tensors taken for the current device's, in front of a library that does nothing."""
    lib._current_device()
    monkeypatch.setattr(lib, "_get_device", lambda: -1)
    monkeypatch.setattr(lib, "lib", _Reached())
    return lib


M, N, K = 4, 32, 64
WIDTH = {torch.bfloat16: [torch.float16], torch.float32: [torch.int32, torch.uint32], torch.float8_e4m3fn:
         [torch.float8_e5m2, torch.float8_e4m3fnuz, torch.float8_e5m2fnuz, torch.int8, torch.bool]}
BITS = {torch.bfloat16: [torch.int16, torch.uint16], torch.float32: [], torch.float8_e4m3fn: [torch.uint8]}


def _calls(lib):  # noqa: F811
    """Every function with tensors of the types it takes: (function, arguments)."""
    def t(*s, d=torch.bfloat16):
        return torch.zeros(*s, dtype=d)

    def f(*s):
        return torch.zeros(*s)

    def e(*s):
        return t(*s, d=torch.float8_e4m3fn)

    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    return [
        (lib.qffn_layernorm_absmax, [t(M, K), t(M, K), f(M), f(M), f(2), t(M, K), t(M, K), t(K), t(K), 1e-5, M, K]),
        (lib.qffn_layernorm_backward, [t(M, K), f(K), f(K), f(2), t(M, K), t(M, K), t(M, K), f(M), f(M), t(K), M, K, False, ws]),
        (lib.qffn_rmsnorm_backward, [t(M, K), f(K), f(2), t(M, K), t(M, K), t(M, K), f(M), t(K), M, K, False, ws]),
        (lib.qffn_linear, [t(M, N), t(M, N), t(M, K), t(N, K), t(N), t(M, N), 2, M, N, K, ws]),
        (lib.qffn_linear_fp8, [t(M, N), t(M, N), e(M, K), f(1), e(N, K), f(1), t(N), t(M, N), 2, M, N, K, ws]),
        (lib.qffn_linear_backward, [t(M, K), t(N, K), f(N), t(M, N), t(M, N), t(M, K), t(N, K), 2, M, N, K, False, ws]),
        (lib.qffn_gated_linear, [t(M, N), t(M, K), t(2 * N, K), 4, M, K, N, ws]),
        (lib.qffn_gated_linear_backward, [t(M, K), t(2 * N, K), t(M, N), t(M, K), t(2 * N, K), 4, M, K, N, False, ws]),
    ]


def test_types_of_the_right_width_are_refused(on_cpu):
    """fp16 is not bf16, int32 not fp32, E5M2 not E4M3: refused for every tensor of every function.  Raw bits
    (int16 and uint16 for bf16, uint8 for E4M3), as the other functions take them, stay."""
    for f, args in _calls(on_cpu):
        f(*args, stream=0)
        for i, a in enumerate(args[:-1]):                           # (the last is the workspace, or a number)
            if not isinstance(a, torch.Tensor):
                continue
            for d in BITS[a.dtype]:
                f(*args[:i], a.view(d), *args[i + 1:], stream=0)
            for d in WIDTH[a.dtype]:
                n = on_cpu.lib.calls
                with pytest.raises(on_cpu.QffnError) as e:
                    f(*args[:i], torch.zeros(a.shape, dtype=torch.uint8).to(d) if d.itemsize == 1 else a.view(d),
                      *args[i + 1:], stream=0)
                assert e.value.status == 1 and on_cpu.lib.calls == n and str(d) in str(e.value), (f.__name__, i, d)


def test_workspace_bytes_limit_the_workspace(on_cpu, monkeypatch):
    """workspace_bytes counts where it is less than the tensor holds, never as more; a negative one is refused."""
    seen = []
    monkeypatch.setattr(on_cpu.lib, "qffn_gated_linear", lambda *a: seen.append(a[8]) or 0)
    f, args = next(c for c in _calls(on_cpu) if c[0].__name__ == "qffn_gated_linear")
    size = args[-1].numel()
    for given, counted in ((None, size), (0, 0), (100, 100), (size, size), (size + 1, size)):
        f(*args, workspace_bytes=given, stream=0)
        assert seen[-1] == counted
    for ws in (args[-1], A):
        with pytest.raises(on_cpu.QffnError) as e:
            f(*args[:-1], ws, workspace_bytes=-1, stream=0)
        assert e.value.status == 1 and len(seen) == 5
