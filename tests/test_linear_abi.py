"""Checks of the norm, linear and gated entry points that need no GPU: refusals before anything is
enqueued, workspace sizes, and the 64-bit plain forms against differences."""
import math

import pytest
import torch

import plain_ops as P
from test_abi import A, MIS, NULL, lib  # noqa: F401  (lib: the module's build-and-load fixture)

ODD4 = A + 2            # below an fp32 pointer's alignment


def _refuses(f, good, wrong):
    """Every (position, value, status) of ``wrong`` put into ``good`` is refused with that status."""
    for i, v, st in wrong:
        args = list(good)
        args[i] = v
        assert f(*args) == st, (i, v, st)


def test_layernorm_refusals(lib):  # noqa: F811
    # res_out, y, mean, rstd, stats, res_in, x, gain, shift, eps, N, C, stream
    good = [A] * 9 + [1e-5, 4, 256, None]
    _refuses(lib.lib.qffn_layernorm_absmax, good,
             [(i, NULL, 1) for i in (0, 1, 2, 3, 6, 7)]            # (res_out: with res_in given)
             + [(9, -1.0, 1), (9, float("nan"), 1), (9, float("inf"), 1), (10, -1, 1), (11, -8, 1)]
             + [(11, 12, 2), (11, 0, 2), (11, 16392, 2), (10, 1 << 31, 2)]
             + [(i, MIS, 3) for i in (0, 1, 5, 6, 7, 8)] + [(i, ODD4, 3) for i in (2, 3, 4)])


def test_norm_backward_refusals(lib):  # noqa: F811
    size = lib.qffn_norm_backward_workspace_size(100, 512)
    assert size >= 256 and size % 256 == 0
    assert lib.qffn_norm_backward_workspace_size(4, 12) == 0 and lib.qffn_norm_backward_workspace_size(-1, 64) == 0
    assert lib.qffn_norm_backward_workspace_size(0, 64) >= 256
    # dx, dgain, dshift, stats, dy, dres, r, mean, rstd, gain, N, C, accumulate, workspace, bytes, stream
    good = [A] * 10 + [100, 512, 0, A, size, None]
    _refuses(lib.lib.qffn_layernorm_backward, good,
             [(i, NULL, 1) for i in (0, 1, 4, 6, 7, 8, 9, 13)] + [(14, size - 1, 1), (10, -1, 1)]
             + [(11, 20, 2), (11, 16392, 2)] + [(i, MIS, 3) for i in (0, 4, 5, 6, 9)]
             + [(i, ODD4, 3) for i in (1, 2, 3, 7, 8)] + [(13, A + 16, 3)])
    # dx, dgain, stats, dy, dres, r, rstd, gain, N, C, accumulate, workspace, bytes, stream
    good = [A] * 8 + [100, 512, 0, A, size, None]
    _refuses(lib.lib.qffn_rmsnorm_backward, good,
             [(i, NULL, 1) for i in (0, 1, 3, 5, 6, 7, 11)] + [(12, size - 1, 1), (8, -1, 1), (9, 20, 2)]
             + [(i, MIS, 3) for i in (0, 3, 4, 5, 7)] + [(i, ODD4, 3) for i in (1, 2, 6)] + [(11, A + 16, 3)])


def test_linear_refusals(lib):  # noqa: F811
    size = lib.qffn_linear_workspace_size(300, 512, 8192)
    assert size > 256                                               # K is split: there are partial sums
    # out, z, x, w, bias, residual, act, M, N, K, workspace, bytes, stream
    good = [A] * 6 + [2, 300, 512, 8192, A, size, None]
    _refuses(lib.lib.qffn_linear, good,
             [(i, NULL, 1) for i in (0, 2, 3, 10)] + [(6, 5, 1), (6, -1, 1), (11, size - 1, 1), (7, -1, 1)]
             + [(8, 12, 2), (8, 0, 2), (9, 4, 2), (9, 0, 2), (7, (1 << 30) + 1, 2), (8, (1 << 20) + 8, 2), (9, (1 << 20) + 8, 2)]
             + [(i, MIS, 3) for i in range(6)] + [(10, A + 16, 3)])
    for bad in ((-1, 8, 8), (8, 12, 8), (8, 8, 12), (8, 0, 8), (8, 8, 0), (1 << 30, 1 << 20, 8)):
        assert lib.qffn_linear_workspace_size(*bad) == 0, bad
    size = lib.qffn_linear_fp8_workspace_size(40, 512, 8192)
    # out, z, x, x_scale, w, w_scale, bias, residual, act, M, N, K, workspace, bytes, stream
    good = [A] * 8 + [0, 40, 512, 8192, A, size, None]
    _refuses(lib.lib.qffn_linear_fp8, good,
             [(i, NULL, 1) for i in (0, 2, 3, 4, 5, 12)] + [(8, 7, 1), (13, size - 1, 1), (9, -1, 1)]
             + [(11, 8200, 2), (10, 20, 2)] + [(i, MIS, 3) for i in (0, 1, 2, 4, 6, 7)]
             + [(i, ODD4, 3) for i in (3, 5)] + [(12, A + 16, 3)])
    assert lib.qffn_linear_fp8_workspace_size(40, 512, 8200) == 0   # K % 16


def test_linear_backward_refusals(lib):  # noqa: F811
    size = lib.qffn_linear_backward_workspace_size(300, 512, 1024)
    # dx, dw, dbias, dout, z, x, w, act, M, N, K, accumulate, workspace, bytes, stream
    good = [A] * 7 + [2, 300, 512, 1024, 0, A, size, None]
    f = lib.lib.qffn_linear_backward
    _refuses(f, good,
             [(i, NULL, 1) for i in (1, 3, 4, 5, 6, 12)] + [(7, 9, 1), (13, size - 1, 1), (8, -1, 1)]
             + [(9, 20, 2), (10, 20, 2), (10, 0, 2)] + [(i, MIS, 3) for i in (0, 1, 3, 4, 5, 6)]
             + [(2, ODD4, 3), (12, A + 16, 3)])
    assert lib.qffn_linear_backward_workspace_size(4, 12, 8) == 0
    assert lib.qffn_linear_backward_workspace_size(1 << 30, 8, 1 << 20) == 0     # dx: too many tiles
    none = list(good)
    none[7], none[4], none[12] = 0, NULL, NULL                      # z is not needed: the next check refuses
    assert f(*none) == 1
    none[12] = A + 16
    assert f(*none) == 3


def test_gated_refusals(lib):  # noqa: F811
    size = lib.qffn_gated_linear_workspace_size(300, 8192, 256)
    assert size > 256
    # h, x, w1, act, N, C, H, workspace, bytes, stream
    good = [A] * 3 + [4, 300, 8192, 256, A, size, None]
    _refuses(lib.lib.qffn_gated_linear, good,
             [(i, NULL, 1) for i in (0, 1, 2, 7)] + [(3, 5, 1), (4, -1, 1), (8, size - 1, 1)]
             + [(5, 12, 2), (6, 12, 2), (6, 0, 2), (6, (1 << 19) + 8, 2)] + [(i, MIS, 3) for i in range(3)] + [(7, A + 16, 3)])
    size = lib.qffn_gated_linear_backward_workspace_size(300, 1024, 256)
    assert size >= 300 * 512 * 2
    # dx, dw1, dh, x, w1, act, N, C, H, accumulate, workspace, bytes, stream
    good = [A] * 5 + [4, 300, 1024, 256, 0, A, size, None]
    _refuses(lib.lib.qffn_gated_linear_backward, good,
             [(i, NULL, 1) for i in (1, 2, 3, 4, 10)] + [(5, -1, 1), (11, size - 1, 1), (6, -1, 1)]
             + [(7, 12, 2), (8, 12, 2)] + [(i, MIS, 3) for i in range(5)] + [(10, A + 16, 3)])
    for bad in ((-1, 8, 8), (4, 12, 8), (4, 8, 12), (4, 8, 1 << 20)):
        assert lib.qffn_gated_linear_workspace_size(*bad) == 0 and lib.qffn_gated_linear_backward_workspace_size(*bad) == 0


def test_workspace_sizes_grow_with_the_call_only(lib):  # noqa: F811
    """They need no device, and a larger call never asks for less than its own buffers."""
    for M in (0, 1, 16, 17, 64, 129, 300, 5000):
        for N, K in ((8, 8), (512, 8192), (4096, 1024)):
            s = lib.qffn_linear_backward_workspace_size(M, N, K)
            assert s >= max(256, M * N * 2) and s % 256 == 0
            g = lib.qffn_gated_linear_backward_workspace_size(M, K, N)
            assert g >= max(256, M * 2 * N * 2) and g % 256 == 0
            assert lib.qffn_linear_workspace_size(M, N, K) >= 256


def test_binding_refuses_tensors(lib):  # noqa: F811
    """Too small, not contiguous, of another width or not on the current device: refused with the
    invalid-argument status before the call."""
    bf = torch.bfloat16
    x, w, out = torch.zeros(4, 64, dtype=bf), torch.zeros(32, 64, dtype=bf), torch.zeros(4, 32, dtype=bf)
    ws = torch.zeros(4096, dtype=torch.uint8)

    def call(x=x, w=w, out=out, ws=ws, M=4):
        lib.qffn_linear(out, None, x, w, None, None, 0, M, 32, 64, ws, stream=0)

    for kw in (dict(x=x[:, ::2]), dict(w=w.float()), dict(out=out[:3]), dict(M=5), dict(x=x.t()), dict(x=x)):
        with pytest.raises(lib.QffnError) as e:                     # (the last: not on a GPU)
            call(**kw)
        assert e.value.status == 1
    with pytest.raises(lib.QffnError) as e:
        lib.qffn_linear(A, None, A, A, None, None, 9, 4, 32, 64, A, 4096, stream=0)
    assert e.value.status == 1
    with pytest.raises(lib.QffnError) as e:
        lib.qffn_layernorm_absmax(None, A, A, A, None, None, A, A, None, 1e-5, 4, 12, stream=0)
    assert e.value.status == 2


@pytest.mark.parametrize("name", list(P.ACTS))
def test_plain_activation_slopes_against_differences(name):
    z = torch.linspace(-6, 6, 241, dtype=torch.float64) + 1e-3      # (off relu's corner)
    h = 1e-5
    d = (P.act(z + h, name) - P.act(z - h, name)) / (2 * h)
    # a central difference is off by h^2 / 6 times the third derivative (below 3) and eps |f| / h
    assert torch.allclose(P.act_grad(z, name), d, rtol=0, atol=3 * h * h + 7 * 2.3e-16 / h * 2)


@pytest.mark.parametrize("centred", [False, True])
def test_plain_norm_backward_against_differences(centred):
    g = torch.Generator().manual_seed(1)
    r, gain, dy, dres = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((3, 16), (16,), (3, 16), (3, 16)))
    eps = 1e-5

    def loss(r, gain, shift):
        if centred:
            y = P.layernorm(r, gain, shift, eps)[0]
        else:
            y = r / torch.sqrt((r * r).mean(1, keepdim=True) + eps) * gain
        return (y * dy).sum() + (r * dres).sum()

    shift = torch.zeros(16, dtype=torch.float64)
    mean = r.mean(1) if centred else None
    rstd = 1 / torch.sqrt(((r - (mean[:, None] if centred else 0)) ** 2).mean(1) + eps)
    dx, dg, ds, _, _, _ = P.norm_backward(dy, dres, r, mean, rstd, gain)
    h = 1e-5
    for t, grad in ((r, dx), (gain, dg), (shift, ds)):
        if t is shift and not centred:
            continue
        flat = t.view(-1)
        for i in range(0, flat.numel(), 5):
            keep = flat[i].item()
            flat[i] = keep + h
            up = loss(r, gain, shift)
            flat[i] = keep - h
            down = loss(r, gain, shift)
            flat[i] = keep
            # cubic terms are below 100 here; the loss is of size 100 at most
            assert math.isclose(grad.view(-1)[i].item(), ((up - down) / (2 * h)).item(), rel_tol=1e-6, abs_tol=100 * h * h + 1e-9)


@pytest.mark.parametrize("name", ["gelu", "silu", "gelu_tanh"])
def test_plain_products_against_differences(name):
    g = torch.Generator().manual_seed(2)
    x, w, w1, d, b = (torch.randn(*s, generator=g, dtype=torch.float64) for s in ((3, 8), (5, 8), (10, 8), (3, 5), (5,)))

    def lin():
        return (P.act(x @ w.t() + b, name) * d).sum()

    def gat():
        return (P.gated(x, w1, name)[0] * d).sum()

    z = x @ w.t() + b
    dx, dw, db, _, _, _ = P.linear_backward(d, z, x, w, name)
    _, _, gdx, gdw, _, _ = P.gated_backward(d, x, w1, name)
    h = 1e-5
    for f, t, grad in ((lin, x, dx), (lin, w, dw), (lin, b, db), (gat, x, gdx), (gat, w1, gdw)):
        flat = t.view(-1)
        for i in range(0, flat.numel(), 3):
            keep = flat[i].item()
            flat[i] = keep + h
            up = f()
            flat[i] = keep - h
            down = f()
            flat[i] = keep
            assert math.isclose(grad.reshape(-1)[i].item(), ((up - down) / (2 * h)).item(), rel_tol=1e-6, abs_tol=1000 * h * h + 1e-9)
