"""Calls without rows: the buffers that have none may be NULL, which is the address of an empty tensor."""
import torch

from test_abi import A, NULL, lib  # noqa: F401  (lib: the module's build-and-load fixture)


def test_row_buffers_may_be_null(lib):  # noqa: F811
    C = lib.lib
    assert C.qffn_layernorm_absmax(NULL, NULL, NULL, NULL, NULL, NULL, NULL, A, NULL, 1e-5, 0, 256, None) == 0
    assert C.qffn_layernorm_backward(NULL, A, A, NULL, NULL, NULL, NULL, NULL, NULL, A, 0, 512, 1, A, 1 << 20, None) == 0
    assert C.qffn_rmsnorm_backward(NULL, A, NULL, NULL, NULL, NULL, NULL, A, 0, 512, 1, A, 1 << 20, None) == 0
    assert C.qffn_linear(NULL, NULL, NULL, A, A, NULL, 2, 0, 512, 8192, A, 1 << 20, None) == 0
    assert C.qffn_linear_fp8(NULL, NULL, NULL, A, A, A, A, NULL, 0, 0, 512, 8192, A, 1 << 20, None) == 0
    assert C.qffn_linear_backward(NULL, A, A, NULL, NULL, NULL, A, 2, 0, 512, 1024, 1, A, 1 << 20, None) == 0
    assert C.qffn_gated_linear(NULL, NULL, A, 4, 0, 8192, 256, A, 1 << 20, None) == 0
    assert C.qffn_gated_linear_backward(NULL, A, NULL, NULL, A, 4, 0, 1024, 256, 1, A, 1 << 20, None) == 0


def test_the_others_may_not(lib):  # noqa: F811
    """Gains, weights, their gradients and the workspace are there without rows too."""
    C = lib.lib
    assert C.qffn_layernorm_absmax(NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, NULL, 1e-5, 0, 256, None) == 1
    for i in (1, 9, 13):
        good = [NULL, A, A, NULL, NULL, NULL, NULL, NULL, NULL, A, 0, 512, 1, A, 1 << 20, None]
        good[i] = NULL
        assert C.qffn_layernorm_backward(*good) == 1, i
    for i in (3, 10):
        good = [NULL, NULL, NULL, A, A, NULL, 2, 0, 512, 8192, A, 1 << 20, None]
        good[i] = NULL
        assert C.qffn_linear(*good) == 1, i
    for i in (1, 6, 12):
        good = [NULL, A, A, NULL, NULL, NULL, A, 2, 0, 512, 1024, 1, A, 1 << 20, None]
        good[i] = NULL
        assert C.qffn_linear_backward(*good) == 1, i
    # and a row that is there needs its buffers
    assert C.qffn_linear(NULL, NULL, A, A, A, NULL, 2, 1, 512, 8192, A, 1 << 20, None) == 1
    assert C.qffn_linear(NULL, NULL, NULL, A, A, NULL, 2, -1, 512, 8192, A, 1 << 20, None) == 1


def test_empty_tensors_through_the_binding(lib):  # noqa: F811
    """Where a batch is empty its tensors are, on whatever device; addresses stand for the rest here."""
    x, out = torch.empty(0, 64, dtype=torch.bfloat16), torch.empty(0, 32, dtype=torch.bfloat16)
    f = torch.empty(0)
    lib.qffn_linear(out, out, x, A, None, out, lib.QFFN_ACT_GELU, 0, 32, 64, A, 1 << 16, stream=0)
    lib.qffn_gated_linear(out, x, A, lib.QFFN_ACT_SILU, 0, 64, 32, A, 1 << 16, stream=0)
    lib.qffn_layernorm_absmax(x, x, f, f, None, x, x, A, None, 1e-5, 0, 64, stream=0)
    lib.qffn_linear_backward(x, A, A, out, out, x, A, lib.QFFN_ACT_GELU, 0, 32, 64, True, A, 1 << 16, stream=0)
