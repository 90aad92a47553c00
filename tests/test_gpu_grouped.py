"""Block-scaled E4M3 products and products grouped by expert against the 64-bit plain forms."""
import pytest
import torch

import plain_blocks as B
import plain_ops as P

pytestmark = pytest.mark.gpu
bf16, u8 = torch.bfloat16, torch.uint8


@pytest.fixture(scope="module")
def q():
    import transformer_ffn_block_gb300 as q
    return q


def _t(seed, *shape, std=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(bf16)


def _wide(seed, *shape):
    """Rows, and parts of 128 of a row, of very different sizes: every scale is another."""
    g = torch.Generator().manual_seed(seed)
    t = torch.randn(*shape, generator=g)
    p = torch.exp2(torch.randint(-8, 8, shape[:-1] + (-(-shape[-1] // 128),), generator=g).float())
    return (t * p.repeat_interleave(128, -1)[..., :shape[-1]]).to(bf16)


def _records(q, x, by):
    """Device codes and scales of a bf16 tensor, and the values they stand for."""
    d = x.cuda()
    if by == 1:
        rows, cols = x.shape
        c, s = torch.empty(rows, cols, dtype=u8, device="cuda"), torch.empty(rows, -(-cols // 128), dtype=u8, device="cuda")
        q.qffn_quantize_blocks(c, s, d, rows, cols)
        return c, s, B.values(c.cpu(), s.cpu())
    n, rows, cols = x.shape
    c = torch.empty(n, rows, cols, dtype=u8, device="cuda")
    s = torch.empty(n, -(-rows // 128), -(-cols // 128), dtype=u8, device="cuda")
    q.qffn_quantize_weight_blocks(c, s, d, n, rows, cols)
    return c, s, torch.stack([B.values(c[i].cpu(), s[i].cpu(), 128) for i in range(n)])


def _new(*shape):
    return torch.full(shape, float("nan"), dtype=bf16, device="cuda")


# rows from one token to a few tiles, columns and K that end inside a tile, a block or a 16-byte load
LINEAR = [(1, 8, 16), (1, 136, 272), (1, 4096, 1024), (2, 1000, 4096), (7, 264, 144), (8, 512, 2048), (9, 256, 128), (16, 1000, 1040),
          (17, 640, 528), (31, 128, 4096), (33, 264, 256), (64, 1000, 2064), (100, 2048, 1024), (128, 384, 8192), (129, 1032, 384),
          (200, 4096, 512), (224, 256, 640), (225, 520, 1152), (300, 2056, 1040), (513, 264, 2048), (1000, 1032, 784), (1400, 4104, 144)]


@pytest.mark.parametrize("M,N,K", LINEAR)
@pytest.mark.parametrize("extras", [False, True])
def test_linear_blocks(q, M, N, K, extras):
    x, xs, xv = _records(q, _wide(M + K, M, K), 1)
    w, ws, wv = _records(q, _wide(N, 1, N, K), 128)
    bias, res = (_t(3, N), _t(4, M, N, std=4.0)) if extras else (None, None)
    out = _new(M, N)
    q.qffn_linear_fp8_blocks(out, x, xs, w, ws, bias.cuda() if extras else None, res.cuda() if extras else None, M, N, K)
    q.qffn_check_status()
    want, bound = B.linear(xv, wv[0], bias.double() if extras else None, res.double() if extras else None)
    P.check(out, want, bound, "out")
    if extras:                                                      # in the place of the residual: the same bits
        again = res.cuda()
        q.qffn_linear_fp8_blocks(again, x, xs, w, ws, bias.cuda(), again, M, N, K)
        assert torch.equal(again, out)


@pytest.mark.parametrize("M", [1, 20, 100, 300])
def test_linear_blocks_special_values(q, M):
    """A NaN code or scale reaches its own row (of x) or column block (of w) alone; the smallest and the largest scales
    multiply as their exponents add."""
    N, K = 264, 400
    x, xs, _ = _records(q, _t(1, M, K), 1)
    w, ws, _ = _records(q, _t(2, 1, N, K), 128)
    base = _new(M, N)
    q.qffn_linear_fp8_blocks(base, x, xs, w, ws, None, None, M, N, K)
    a, b = xs.clone(), ws.clone()
    a[M // 2, 1], b[0, 1, 3] = 255, 255
    out = _new(M, N)
    q.qffn_linear_fp8_blocks(out, x, a, w, b, None, None, M, N, K)
    want = base.clone()
    want[M // 2], want[:, 128:256] = float("nan"), float("nan")
    assert torch.equal(torch.isnan(out), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(out), torch.nan_to_num(want))
    for up in (90, -90):
        q.qffn_linear_fp8_blocks(out, x, (xs.int() + up).to(u8), w, (ws.int() - up).to(u8), None, None, M, N, K)
        assert torch.equal(out, base)


def _sizes(kind, G, M):
    g = torch.Generator().manual_seed(G + M)
    if kind == "ragged":
        s = torch.bincount((torch.rand(M, generator=g) ** 2 * G).long().clamp_max(G - 1), minlength=G)
    elif kind == "one":                                             # all rows in one group, the others empty
        s = torch.zeros(G, dtype=torch.long)
        s[G // 2] = M
    else:                                                           # every third group empty, rows before and behind
        s = torch.bincount(torch.randint(0, G, (max(M - 5, 0),), generator=g) // 3 * 3, minlength=G)[:G]
    o = torch.cat([torch.zeros(1, dtype=torch.long), s.cumsum(0)])
    if kind == "gaps" and M > 5:
        o = o + 2
    return o.to(torch.int32)


GROUPED = [(1, 1, 8, 16), (1, 300, 264, 272), (3, 1, 1000, 144), (8, 2, 512, 4096), (5, 7, 136, 1040), (8, 16, 1032, 512), (16, 33, 264, 256),
           (4, 100, 2048, 1024), (64, 200, 264, 528), (3, 500, 520, 1152), (8, 900, 1032, 784), (2, 1500, 256, 2064), (130, 700, 136, 144),
           (300, 40, 264, 272), (1000, 3000, 72, 80)]


@pytest.mark.parametrize("G,M,N,K", GROUPED)
@pytest.mark.parametrize("kind", ["ragged", "one", "gaps"])
@pytest.mark.parametrize("fp8", [False, True])
def test_grouped(q, G, M, N, K, kind, fp8):
    off = _sizes(kind, G, M)
    out = _new(M, N)
    if fp8:
        x, xs, xv = _records(q, _wide(M, M, K), 1)
        w, ws, wv = _records(q, _wide(N, G, N, K), 128)
        q.qffn_grouped_linear_fp8_blocks(out, x, xs, w, ws, off.cuda(), G, M, N, K)
    else:
        hx, hw = _t(M, M, K), _t(N, G, N, K, std=0.1)
        xv, wv = hx.double(), hw.double()
        q.qffn_grouped_linear(out, hx.cuda(), hw.cuda(), off.cuda(), G, M, N, K)
    q.qffn_check_status()
    want, bound, live = B.grouped(xv, wv, off)
    P.check(out[live.cuda()], want[live], bound[live], "out")
    assert bool(torch.isnan(out[~live.cuda()]).all())               # left as they were


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("M", [6, 40, 700])
def test_grouped_neighbours_do_not_mix(q, M, fp8):
    """Infinities and NaN in one group's rows and matrix stay in that group, also where its rows, columns or K end inside a
    tile, and so do those in rows of no group."""
    G, N, K = 4, 200, 208
    off = torch.tensor([1, M // 4 + 1, M // 2, M // 2, M - 1], dtype=torch.int32)
    x, w = _t(1, M, K), _t(2, G, N, K)
    bad = slice(int(off[1]), int(off[2]))
    args = lambda x, w: ((*_records(q, x, 1)[:2], *_records(q, w, 128)[:2]) if fp8 else (x.cuda(), w.cuda()))  # noqa: E731
    call = q.qffn_grouped_linear_fp8_blocks if fp8 else q.qffn_grouped_linear
    base, out = _new(M, N), _new(M, N)
    call(base, *args(x, w), off.cuda(), G, M, N, K)
    x[bad], w[1] = float("nan"), float("inf")
    x[0], x[-1], w[2] = float("inf"), float("nan"), float("nan")   # rows of no group; the matrix of an empty one
    call(out, *args(x, w), off.cuda(), G, M, N, K)
    q.qffn_check_status()
    want = base.clone()
    want[bad] = float("nan")
    assert torch.equal(torch.nan_to_num(out, nan=7.0), torch.nan_to_num(want, nan=7.0))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("M", [10, 400])
def test_offsets_outside_the_rows_are_clamped(q, M, fp8):
    G, N, K = 4, 72, 144
    off = torch.tensor([-7, M // 3, M // 3 - 2, M // 2, M + 1000], dtype=torch.int32)     # group 1 has no rows, group 2 two more
    x, w = _t(1, M, K), _t(2, G, N, K)
    guard = torch.full((M + 64, N), 3.0, dtype=bf16, device="cuda")
    out = guard[:M]
    if fp8:
        x, xs, xv = _records(q, x, 1)
        w, ws, wv = _records(q, w, 128)
        q.qffn_grouped_linear_fp8_blocks(out, x, xs, w, ws, off.cuda(), G, M, N, K)
    else:
        xv, wv = x.double(), w.double()
        q.qffn_grouped_linear(out, x.cuda(), w.cuda(), off.cuda(), G, M, N, K)
    q.qffn_check_status()
    assert bool((guard[M:] == 3.0).all())
    want, bound, _ = B.grouped(xv, wv, [0, M // 3, M // 3, M // 2, M])
    sure = [i for i in range(M) if not M // 3 - 2 <= i < M // 3]    # (rows that two groups claim are undefined)
    P.check(out[sure], want[sure], bound[sure], "out")


@pytest.mark.parametrize("G,M,N,K", GROUPED)
@pytest.mark.parametrize("kind", ["ragged", "one", "gaps"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_grouped_backward(q, G, M, N, K, kind, accumulate):
    off = _sizes(kind, G, M)
    dout, x, w = _t(1, M, N, std=0.1), _t(2, M, K), _t(3, G, N, K, std=0.1)
    old = _t(4, G, N, K) if accumulate else None
    dx, dw = _new(M, K), old.cuda() if accumulate else _new(G, N, K)
    q.qffn_grouped_linear_backward(dx, dw, dout.cuda(), x.cuda(), w.cuda(), off.cuda(), G, M, N, K, accumulate)
    q.qffn_check_status()
    want_dx, want_dw, b_dx, b_dw, live = B.grouped_backward(dout.double(), x.double(), w.double(), off,
                                                            old.double() if accumulate else None)
    P.check(dx[live.cuda()], want_dx[live], b_dx[live], "dx")
    P.check(dw, want_dw, b_dw, "dw")
    assert bool(torch.isnan(dx[~live.cuda()]).all())                # left as they were
    again = old.cuda() if accumulate else _new(G, N, K)             # the weight gradient alone, the same bits
    q.qffn_grouped_linear_backward(None, again, dout.cuda(), x.cuda(), w.cuda(), off.cuda(), G, M, N, K, accumulate)
    assert torch.equal(again, dw)


@pytest.mark.parametrize("M", [6, 40, 700])
def test_grouped_backward_neighbours_do_not_mix(q, M):
    """A group that ends anywhere: what the next one, or no group, holds does not reach its gradients."""
    G, N, K = 4, 200, 208
    off = torch.tensor([1, M // 4 + 1, M // 2, M // 2, M - 1], dtype=torch.int32)
    dout, x, w = _t(1, M, N), _t(2, M, K), _t(3, G, N, K)
    bad = slice(int(off[1]), int(off[2]))

    def run():
        dx, dw = _new(M, K), _new(G, N, K)
        q.qffn_grouped_linear_backward(dx, dw, dout.cuda(), x.cuda(), w.cuda(), off.cuda(), G, M, N, K, False)
        q.qffn_check_status()
        return dx, dw

    base_dx, base_dw = run()
    dout[bad], w[1] = float("nan"), float("inf")
    for t in (x, dout):
        t[0], t[-1] = float("inf"), float("nan")
    x[bad], w[2] = float("-inf"), float("nan")
    dx, dw = run()
    base_dx[bad], base_dw[1] = float("nan"), float("nan")
    for got, want in ((dx, base_dx), (dw, base_dw)):
        assert torch.equal(torch.nan_to_num(got, nan=7.0), torch.nan_to_num(want, nan=7.0))
    assert not dw[2].any()
