"""Checks of the block-scaled and grouped entry points that need no GPU: refusals before anything is enqueued, the
binding's checks of tensors, and the plain forms against other ways to the same values."""
import pytest
import torch

import brute
import plain_blocks as B
from test_abi import A, MIS, NULL, lib  # noqa: F401  (lib: the module's build-and-load fixture)
from test_linear_abi import ODD4, _refuses


def test_quantize_refusals(lib):  # noqa: F811
    # q, scale, in, rows, cols, stream (scales have no alignment)
    good = [A, A + 1, A, 4, 256, None]
    _refuses(lib.lib.qffn_quantize_blocks, good,
             [(i, NULL, 1) for i in (0, 1, 2)] + [(3, -1, 1), (4, -16, 1), (4, 24, 2), (4, 0, 2), (4, (1 << 20) + 16, 2), (3, 1 << 31, 2)]
             + [(0, MIS, 3), (2, MIS, 3)])
    # q, scale, w, count, rows, cols, stream
    good = [A, A + 1, A, 2, 4, 256, None]
    _refuses(lib.lib.qffn_quantize_weight_blocks, good,
             [(i, NULL, 1) for i in (0, 1, 2)] + [(3, -1, 1), (4, -1, 1), (5, 40, 2), (3, 4097, 2), (0, MIS, 3), (2, MIS, 3)])
    # res_out, y, q, scale, rstd, res_in, x, gain, eps, N, C, stream
    good = [A] * 8 + [1e-5, 4, 256, None]
    _refuses(lib.lib.qffn_rmsnorm_quantize_blocks, good,
             [(i, NULL, 1) for i in (0, 2, 3, 4, 6, 7)] + [(8, -1.0, 1), (8, float("nan"), 1), (9, -1, 1), (10, 24, 2), (10, 16400, 2)]
             + [(i, MIS, 3) for i in (0, 1, 2, 5, 6, 7)] + [(4, ODD4, 3)])
    # h, q, scale, gate_up, N, H, stream
    good = [A, A, A + 1, A, 4, 256, None]
    _refuses(lib.lib.qffn_swiglu_quantize_blocks, good,
             [(i, NULL, 1) for i in (1, 2, 3)] + [(4, -1, 1), (5, 8, 2), (5, 40, 2)] + [(i, MIS, 3) for i in (0, 1, 3)])


def test_product_refusals(lib):  # noqa: F811
    # out, x, x_scale, w, w_scale, bias, residual, M, N, K, stream
    good = [A, A, A + 1, A, A + 1, A, A, 4, 256, 512, None]
    _refuses(lib.lib.qffn_linear_fp8_blocks, good,
             [(i, NULL, 1) for i in (0, 1, 2, 3, 4)] + [(7, -1, 1), (8, 12, 2), (8, 0, 2), (9, 24, 2), (9, 0, 2), (7, (1 << 30) + 1, 2)]
             + [(i, MIS, 3) for i in (0, 1, 3, 5, 6)])
    # out, x, w, offsets, G, M, N, K, stream
    good = [A, A, A, A, 8, 4, 256, 512, None]
    _refuses(lib.lib.qffn_grouped_linear, good,
             [(i, NULL, 1) for i in range(4)] + [(4, 0, 1), (4, -1, 1), (4, 4097, 2), (5, -1, 1), (6, 12, 2), (7, 12, 2), (7, 0, 2)]
             + [(i, MIS, 3) for i in range(3)] + [(3, ODD4, 3)])
    # dx, dw, dout, x, w, offsets, G, M, N, K, accumulate, stream
    good = [A] * 6 + [8, 4, 256, 512, 0, None]
    _refuses(lib.lib.qffn_grouped_linear_backward, good,
             [(i, NULL, 1) for i in (1, 2, 3, 4, 5)] + [(6, 0, 1), (6, 4097, 2), (7, -1, 1), (8, 12, 2), (9, 12, 2), (8, 0, 2)]
             + [(i, MIS, 3) for i in range(5)] + [(5, ODD4, 3)])
    big = list(good)
    big[6], big[8], big[9] = 4096, 1 << 17, 1 << 17                 # dw of 2^30 tiles
    assert lib.lib.qffn_grouped_linear_backward(*big) == 2
    # out, x, x_scale, w, w_scale, offsets, G, M, N, K, stream
    good = [A, A, A + 1, A, A + 1, A, 8, 4, 256, 512, None]
    _refuses(lib.lib.qffn_grouped_linear_fp8_blocks, good,
             [(i, NULL, 1) for i in range(6)] + [(6, 0, 1), (6, 4097, 2), (7, -1, 1), (8, 12, 2), (9, 24, 2)]
             + [(i, MIS, 3) for i in (0, 1, 3)] + [(5, ODD4, 3)])


def test_calls_without_rows(lib):  # noqa: F811
    """Empty tensors have no address; nothing is enqueued for them."""
    f = lib.lib
    assert f.qffn_quantize_blocks(NULL, NULL, NULL, 0, 256, None) == 0
    assert f.qffn_quantize_weight_blocks(NULL, NULL, NULL, 0, 128, 256, None) == 0
    assert f.qffn_quantize_weight_blocks(NULL, NULL, NULL, 3, 0, 256, None) == 0
    assert f.qffn_rmsnorm_quantize_blocks(NULL, NULL, NULL, NULL, NULL, A, NULL, A, 1e-5, 0, 256, None) == 0
    assert f.qffn_swiglu_quantize_blocks(NULL, NULL, NULL, NULL, 0, 256, None) == 0
    assert f.qffn_linear_fp8_blocks(NULL, NULL, NULL, A, A, NULL, NULL, 0, 256, 512, None) == 0
    assert f.qffn_grouped_linear(NULL, NULL, A, A, 4, 0, 256, 512, None) == 0
    assert f.qffn_grouped_linear_fp8_blocks(NULL, NULL, NULL, A, A, A, 4, 0, 256, 512, None) == 0
    assert f.qffn_grouped_linear_backward(NULL, A, NULL, NULL, A, A, 4, 0, 256, 512, 1, None) == 0


def test_binding_refuses_tensors(lib):  # noqa: F811
    """Of another type, too small, not contiguous or not on the current device."""
    bf, u8 = torch.bfloat16, torch.uint8
    x, w, out = torch.zeros(4, 64, dtype=bf), torch.zeros(2, 32, 64, dtype=bf), torch.zeros(4, 32, dtype=bf)
    off = torch.zeros(3, dtype=torch.int32)

    def grouped(x=x, w=w, out=out, off=off):
        lib.qffn_grouped_linear(out, x, w, off, 2, 4, 32, 64, stream=0)

    for kw in (dict(off=off.long()), dict(off=off[:2]), dict(off=torch.zeros(6, dtype=torch.int32)[::2]), dict(w=w[:1]), dict(x=x.float()),
               dict()):                                             # (the last: not on a GPU)
        with pytest.raises(lib.QffnError) as e:
            grouped(**kw)
        assert e.value.status == 1
    q, s = torch.zeros(4, 64, dtype=torch.float8_e4m3fn), torch.zeros(4, 1, dtype=torch.float8_e8m0fnu)
    wq, ws = torch.zeros(32, 64, dtype=u8), torch.zeros(1, 1, dtype=u8)

    def linear(q=q, s=s, wq=wq, ws=ws, K=64):
        lib.qffn_linear_fp8_blocks(out, q, s, wq, ws, None, None, 4, 32, K, stream=0)

    for kw in (dict(s=torch.ones(4)), dict(s=s[:3]), dict(ws=ws[:0]), dict(q=q.view(torch.int8)), dict(K=256), dict()):
        with pytest.raises(lib.QffnError) as e:
            linear(**kw)
        assert e.value.status == 1
    with pytest.raises(lib.QffnError) as e:
        lib.qffn_quantize_blocks(A, A, A, 4, 24, stream=0)
    assert e.value.status == 2


def test_plain_rounding_is_the_nearest_code():
    """plain_blocks.e4m3 against a search over all codes."""
    g = torch.Generator().manual_seed(1)
    v = torch.cat([torch.randn(400, generator=g).double() * 2.0 ** torch.randint(-12, 8, (400,), generator=g),
                   torch.tensor([0.0, 448.0, -448.0, 1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10, 2.0 ** -9, 15.5, 17.0]).double()])
    v = v.clamp(-448, 448)
    codes = torch.tensor([c for c in range(256) if c & 0x7F != 0x7F], dtype=torch.uint8)
    all_values = codes.view(torch.float8_e4m3fn).float().double()
    got = B.e4m3(v)
    assert torch.equal(got, v.float().to(torch.float8_e4m3fn).float().double())
    assert torch.allclose((got - v).abs(), (all_values[None] - v[:, None]).abs().amin(1), rtol=0, atol=0)
    assert len(brute._E4M3_VALS) == 127                             # the independent table has the same values
    assert sorted(set(all_values.abs().tolist())) == [float(x) for x in brute._E4M3_VALS]


@pytest.mark.parametrize("amax,code", [(0.0, 127), (448.0, 127), (448.5, 128), (224.0, 126), (1.75, 119), (1.76, 120), (2.0 ** -140, 0),
                                       (float("inf"), 255), (3.3e38, 247)])
def test_plain_scale_codes(amax, code):
    assert B.code_of(amax) == code


def test_plain_gradient_against_differences():
    """dx and dw of the grouped products against central differences of sum(out * dout): exact up to rounding, as the
    products are linear in each operand."""
    g = torch.Generator().manual_seed(0)
    off, M, N, K = [0, 3, 3, 7], 8, 3, 4
    x, w, dout = (torch.randn(*s, generator=g).double() for s in ((M, K), (3, N, K), (M, N)))
    dx, dw, _, _, live = B.grouped_backward(dout, x, w, off)
    f = lambda x, w: float((B.grouped(x, w, off)[0] * dout).sum())  # noqa: E731
    h = 0.5
    for t, d in ((x, dx), (w, dw)):
        for i in range(t.numel()):
            e = torch.zeros_like(t).view(-1)
            e[i] = h
            e = e.view_as(t)
            diff = (f(x + e, w) - f(x - e, w)) if t is x else (f(x, w + e) - f(x, w - e))
            assert abs(diff / (2 * h) - d.reshape(-1)[i].item()) < 1e-12 * 100
    assert live.tolist() == [True] * 7 + [False] and not dw[1].any() and not dx[7].any()
