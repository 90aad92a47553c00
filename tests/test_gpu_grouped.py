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
          (200, 4096, 512), (224, 256, 640), (225, 520, 1152), (300, 2056, 1040), (513, 264, 2048), (1000, 1032, 784), (1400, 4104, 144),
          # K over clusters of 8, 4 and 2, two CTAs per SM; one accumulator of 256 rows; several rounds of units
          (40, 256, 16384), (64, 4096, 4096), (130, 4096, 2048), (64, 14336, 528), (1024, 4096, 272), (2500, 2056, 400)]


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
           (300, 40, 264, 272), (1000, 3000, 72, 80),
           # few units of long K: parts of it over clusters of 8, 4 and 2; wide matrices
           (1, 9, 248, 10288), (2, 554, 144, 3840), (2, 84, 1008, 3584), (4, 800, 1024, 4096), (2, 200, 6000, 1040)]


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
def test_offsets_that_are_not_in_order(q, M, fp8):
    """Outside 0 .. M, or below the one before: as the header says, and nothing is written behind the rows."""
    G, N, K = 70, 72, 144
    off = torch.full((G + 1,), M // 2, dtype=torch.int32)
    off[0], off[1], off[2], off[30], off[31], off[33], off[60], off[-1] = -7, M // 3, M // 3 - 2, M // 2 + 3, 0, M // 2 + 1, -1, M + 1000
    x, w = _t(1, M, K), _t(2, G, N, K)
    guard = torch.full((M + 64, N), 3.0, dtype=bf16, device="cuda")
    out = guard[:M]
    if fp8:
        xq, xs, xv = _records(q, x, 1)
        wq, ws, wv = _records(q, w, 128)
        q.qffn_grouped_linear_fp8_blocks(out, xq, xs, wq, ws, off.cuda(), G, M, N, K)
    else:
        xv, wv = x.double(), w.double()
        q.qffn_grouped_linear(out, x.cuda(), w.cuda(), off.cuda(), G, M, N, K)
        dout, dx, dw = _t(3, M, N), _new(M, K), _new(G, N, K)
        q.qffn_grouped_linear_backward(dx, dw, dout.cuda(), x.cuda(), w.cuda(), off.cuda(), G, M, N, K, False)
        want_dx, want_dw, b_dx, b_dw, live = B.grouped_backward(dout.double(), xv, wv, off)
        P.check(dx[live.cuda()], want_dx[live], b_dx[live], "dx")
        P.check(dw, want_dw, b_dw, "dw")
    q.qffn_check_status()
    assert bool((guard[M:] == 3.0).all())
    want, bound, live = B.grouped(xv, wv, off)
    P.check(out[live.cuda()], want[live], bound[live], "out")
    assert bool((out[~live.cuda()] == 3.0).all())


@pytest.mark.parametrize("M", [3, 12, 40, 300])
@pytest.mark.parametrize("blocks", [4, 5])
def test_scales_at_any_address(q, M, blocks):
    """Scales have no alignment: the same bits as with aligned ones."""
    N, K = 264, 128 * blocks
    x, xs, _ = _records(q, _wide(1, M, K), 1)
    w, ws, _ = _records(q, _wide(2, 1, N, K), 128)
    off = torch.tensor([0, M], dtype=torch.int32, device="cuda")
    outs = []
    for shift in (0, 1, 2):
        bx, bw = (torch.zeros(t.numel() + shift, dtype=u8, device="cuda")[shift:] for t in (xs, ws))
        bx.copy_(xs.flatten())
        bw.copy_(ws.flatten())
        one, two = _new(M, N), _new(M, N)
        q.qffn_linear_fp8_blocks(one, x, bx, w, bw, None, None, M, N, K)
        q.qffn_grouped_linear_fp8_blocks(two, x, bx, w, bw, off, 1, M, N, K)
        outs.append((one, two))
    q.qffn_check_status()
    for a, b in outs[1:]:
        assert torch.equal(a, outs[0][0]) and torch.equal(b, outs[0][1])


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


@pytest.mark.parametrize("G,M,N,K", [(1, 3, 8728, 680), (2, 5, 4104, 72), (3, 40, 6152, 136), (1, 1, 16384, 8), (5, 33, 8200, 264)])
@pytest.mark.parametrize("kind", ["ragged", "one", "gaps"])
@pytest.mark.parametrize("accumulate", [False, True])
def test_grouped_backward_of_long_rows(q, G, M, N, K, kind, accumulate):
    """Few rows of dout that are much longer than those of x, written by the kernel just before the call."""
    off = _sizes(kind, G, M)
    dout, x, w = _t(1, M, N, std=0.1), _t(2, M, K), _t(3, G, N, K, std=0.1)
    old = _t(4, G, N, K) if accumulate else None
    d, xs, ws, o = dout.cuda(), x.cuda(), w.cuda(), off.cuda()
    dx, dw = _new(M, K), old.cuda() if accumulate else _new(G, N, K)
    late_d, late_x = torch.zeros_like(d), torch.zeros_like(xs)
    torch.cuda.synchronize()
    late_d.copy_(d)
    late_x.copy_(xs)
    q.qffn_grouped_linear_backward(dx, dw, late_d, late_x, ws, o, G, M, N, K, accumulate)
    then = dx.clone(), dw.clone()                                   # (read by the kernel just behind)
    q.qffn_check_status()
    want_dx, want_dw, b_dx, b_dw, live = B.grouped_backward(dout.double(), x.double(), w.double(), off,
                                                            old.double() if accumulate else None)
    P.check(then[0][live.cuda()], want_dx[live], b_dx[live], "dx")
    P.check(then[1], want_dw, b_dw, "dw")
    assert bool(torch.isnan(dx[~live.cuda()]).all())


@pytest.mark.parametrize("M", [17, 9000])
def test_most_groups(q, M):
    """4096 groups, the most: both products and the gradients, against the group of each row."""
    G, N, K = 4096, 40, 48
    off = _sizes("ragged", G, M)
    x, dout, w = _t(1, M, K), _t(2, M, N, std=0.1), _t(3, G, N, K, std=0.1)
    xq, xs, xv = _records(q, x, 1)
    wq, ws, wv = _records(q, w, 128)
    o, one, two = off.cuda(), _new(M, N), _new(M, N)
    q.qffn_grouped_linear(one, x.cuda(), w.cuda(), o, G, M, N, K)
    q.qffn_grouped_linear_fp8_blocks(two, xq, xs, wq, ws, o, G, M, N, K)
    dx, dw = _new(M, K), _new(G, N, K)
    q.qffn_grouped_linear_backward(dx, dw, dout.cuda(), x.cuda(), w.cuda(), o, G, M, N, K, False)
    q.qffn_check_status()
    want, bound, live = B.grouped(x.double(), w.double(), off)
    P.check(one[live.cuda()], want[live], bound[live], "bf16")
    want, bound, live = B.grouped(xv, wv, off)
    P.check(two[live.cuda()], want[live], bound[live], "E4M3")
    want_dx, want_dw, b_dx, b_dw, live = B.grouped_backward(dout.double(), x.double(), w.double(), off, None)
    P.check(dx[live.cuda()], want_dx[live], b_dx[live], "dx")
    P.check(dw, want_dw, b_dw, "dw")


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


@pytest.mark.parametrize("fp8", [False, True])
def test_matrices_past_two_to_the_31(q, fp8):
    """Only the last of 20 matrices of 2^27 values has rows, and is not zero."""
    G, N, K, M = 20, 1 << 14, 1 << 13, 70
    off = torch.tensor([0] * G + [M], dtype=torch.int32, device="cuda")
    x, last = _wide(1, M, K) if fp8 else _t(1, M, K), _t(2, 1, N, K, std=0.1)
    out, one = _new(M, N), _new(M, N)
    if fp8:
        xq, xs, _ = _records(q, x, 1)
        lq, ls, _ = _records(q, last, 128)
        w = torch.zeros(G, N, K, dtype=u8, device="cuda")
        ws = torch.full((G, N // 128, K // 128), 127, dtype=u8, device="cuda")
        w[-1], ws[-1] = lq[0], ls[0]
        q.qffn_grouped_linear_fp8_blocks(out, xq, xs, w, ws, off, G, M, N, K)
        q.qffn_linear_fp8_blocks(one, xq, xs, lq, ls, None, None, M, N, K)
        rel = 2 * P.HALF + 2 * K * P.ACC                            # the same sums in another order, two roundings
        size = xq.view(torch.float8_e4m3fn).float() * torch.exp2(xs.float() - 127).repeat_interleave(128, 1)
        size = size.abs() @ last[0].cuda().float().abs().t() * 1.07
    else:
        w = torch.zeros(G, N, K, dtype=bf16, device="cuda")
        w[-1] = last[0].cuda()
        q.qffn_grouped_linear(out, x.cuda(), w, off, G, M, N, K)
        q.qffn_grouped_linear(one, x.cuda(), last.cuda(), torch.tensor([0, M], dtype=torch.int32, device="cuda"), 1, M, N, K)
        rel, size = 0.0, torch.zeros(())                            # the same form: the same bits
    q.qffn_check_status()
    assert bool(((out.float() - one.float()).abs() <= rel * size).all())


def test_gradients_past_two_to_the_31(q):
    G, N, K, M = 20, 1 << 14, 1 << 13, 70
    dout, x, last = _t(1, M, N, std=0.1), _t(2, M, K), _t(3, 1, N, K, std=0.1)
    w, dw, dx = torch.zeros(G, N, K, dtype=bf16, device="cuda"), _new(G, N, K), _new(M, K)
    w[-1] = last[0].cuda()
    args = dout.cuda(), x.cuda()
    q.qffn_grouped_linear_backward(dx, dw, *args, w, torch.tensor([0] * G + [M], dtype=torch.int32, device="cuda"), G, M, N, K, False)
    one_dx, one_dw = _new(M, K), _new(1, N, K)
    q.qffn_grouped_linear_backward(one_dx, one_dw, *args, last.cuda(), torch.tensor([0, M], dtype=torch.int32, device="cuda"), 1, M, N, K,
                                   False)
    q.qffn_check_status()
    assert torch.equal(dx, one_dx) and torch.equal(dw[-1], one_dw[0]) and not dw[:-1].any()


def test_rows_past_two_to_the_31(q):
    """An output of more than 2^31 values; the last rows against a call of their own."""
    G, N, K, M = 2, 1 << 16, 64, (1 << 15) + 40
    x, w = torch.zeros(M, K, dtype=bf16, device="cuda"), _t(2, G, N, K).cuda()
    x[-40:] = _t(1, 40, K).cuda()
    out, one = _new(M, N), _new(40, N)
    q.qffn_grouped_linear(out, x, w, torch.tensor([0, M - 40, M], dtype=torch.int32, device="cuda"), G, M, N, K)
    q.qffn_grouped_linear(one, x[-40:].contiguous(), w, torch.tensor([0, 0, 40], dtype=torch.int32, device="cuda"), G, 40, N, K)
    q.qffn_check_status()
    assert torch.equal(out[-40:], one) and not out[:-40].any()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("M", [20, 600])
def test_one_graph_for_other_sizes(q, M, fp8):
    """A captured call reads the offsets when it is replayed; captured beside a backward call."""
    G, N, K = 6, 264, 400
    x, w, dout = _t(1, M, K), _t(2, G, N, K, std=0.1), _t(3, M, N, std=0.1)
    off = torch.zeros(G + 1, dtype=torch.int32, device="cuda")
    out, dx, dw = _new(M, N), _new(M, K), _new(G, N, K)
    dev = [t.cuda() for t in (x, w, dout)]
    if fp8:
        xq, xs, xv = _records(q, x, 1)
        wq, ws, wv = _records(q, w, 128)

    def call():
        if fp8:
            q.qffn_grouped_linear_fp8_blocks(out, xq, xs, wq, ws, off, G, M, N, K)
        else:
            q.qffn_grouped_linear(out, dev[0], dev[1], off, G, M, N, K)
        q.qffn_grouped_linear_backward(dx, dw, dev[2], dev[0], dev[1], off, G, M, N, K, False)

    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for kind in ("ragged", "one", "gaps"):
        o = _sizes(kind, G, M)
        off.copy_(o)
        out.fill_(float("nan"))
        dx.fill_(float("nan"))
        graph.replay()
        q.qffn_check_status()
        want, bound, live = B.grouped(xv if fp8 else x.double(), wv if fp8 else w.double(), o)
        P.check(out[live.cuda()], want[live], bound[live], "out")
        assert bool(torch.isnan(out[~live.cuda()]).all())
        want_dx, want_dw, b_dx, b_dw, live = B.grouped_backward(dout.double(), x.double(), w.double(), o)
        P.check(dx[live.cuda()], want_dx[live], b_dx[live], "dx")
        P.check(dw, want_dw, b_dw, "dw")


def test_two_streams_at_once(q):
    """Calls that overlap have nothing in common (no workspace): the same bits as one after the other."""
    G, M, N, K = 8, 900, 1032, 784
    off = _sizes("ragged", G, M).cuda()
    data = [(_t(10 * i, M, K).cuda(), _t(10 * i + 1, G, N, K, std=0.1).cuda(), _t(10 * i + 2, M, N, std=0.1).cuda()) for i in range(2)]
    rec = [(_records(q, x.cpu(), 1)[:2], _records(q, w.cpu(), 128)[:2]) for x, w, _ in data]

    def run(i, stream):
        x, w, d = data[i]
        out, f8, dx, dw = _new(M, N), _new(M, N), _new(M, K), _new(G, N, K)
        torch.cuda.synchronize()
        for _ in range(5):
            q.qffn_grouped_linear(out, x, w, off, G, M, N, K, stream=stream)
            q.qffn_grouped_linear_backward(dx, dw, d, x, w, off, G, M, N, K, False, stream=stream)
            q.qffn_grouped_linear_fp8_blocks(f8, *rec[i][0], *rec[i][1], off, G, M, N, K, stream=stream)
        return out, f8, dx, dw

    alone = [run(i, None) for i in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    both = [run(i, streams[i]) for i in range(2)]
    torch.cuda.synchronize()
    q.qffn_check_status()
    for a, b in zip(alone, both):
        assert all(torch.equal(s, t) for s, t in zip(a, b))


def test_same_bits_in_every_run(q):
    G, M, N, K = 8, 900, 1032, 784
    off = _sizes("ragged", G, M).cuda()
    x, w, d = _t(1, M, K).cuda(), _t(2, G, N, K, std=0.1).cuda(), _t(3, M, N, std=0.1).cuda()
    first = None
    for _ in range(4):
        out, dx, dw = _new(M, N), _new(M, K), _new(G, N, K)
        q.qffn_grouped_linear(out, x, w, off, G, M, N, K)
        q.qffn_grouped_linear_backward(dx, dw, d, x, w, off, G, M, N, K, False)
        first = first or (out, dx, dw)
        assert all(torch.equal(a, b) for a, b in zip(first, (out, dx, dw)))


# Independent roundings of relative size at most HALF along the way add in the mean square, and no step here
# amplifies them by more than about two: 16 HALF bounds the whole chain (as in test_gpu_blocks.py).
CHAIN = 16 * P.HALF


def _rel(got, want):
    return ((got.double().cpu() - want).norm() / want.norm()).item()


def _route(T, G, top, seed):
    """Routed rows sorted by expert: the token of each, and the offsets."""
    experts = torch.randn(T, G, generator=torch.Generator().manual_seed(seed)).topk(top, dim=1).indices.flatten()
    order = experts.argsort(stable=True)
    sizes = torch.bincount(experts, minlength=G)
    return order // top, torch.cat([torch.zeros(1, dtype=torch.long), sizes.cumsum(0)]).to(torch.int32)


@pytest.mark.parametrize("T,G,top,C,H", [(1, 8, 2, 512, 272), (9, 16, 4, 272, 400), (150, 8, 2, 1024, 640), (700, 4, 2, 528, 1040)])
def test_experts_in_e4m3(q, T, G, top, C, H):
    """r = res + x; y = rms(r) in E4M3; its rows by expert through gate|up, SwiGLU in E4M3 and down: the plain chain with
    the same quantisations."""
    x, res, gain = _t(1, T, C), _t(2, T, C), (torch.randn(C, generator=torch.Generator().manual_seed(3)) * 0.1 + 1).to(bf16)
    w1, w2 = _t(4, G, 2 * H, C, std=C ** -0.5), _t(5, G, C, H, std=H ** -0.5)
    token, off = _route(T, G, top, T)
    M = len(token)
    r, yq, ys, rstd = _new(T, C), torch.empty(T, C, dtype=u8, device="cuda"), torch.empty(T, -(-C // 128), dtype=u8, device="cuda"), torch.empty(T, device="cuda")
    q.qffn_rmsnorm_quantize_blocks(r, None, yq, ys, rstd, res.cuda(), x.cuda(), gain.cuda(), 1e-5, T, C)
    q1, s1, v1 = _records(q, w1, 128)
    q2, s2, v2 = _records(q, w2, 128)
    t = token.cuda()
    gu, out = _new(M, 2 * H), _new(M, C)
    hq, hs = torch.empty(M, H, dtype=u8, device="cuda"), torch.empty(M, -(-H // 128), dtype=u8, device="cuda")
    q.qffn_grouped_linear_fp8_blocks(gu, yq[t], ys[t], q1, s1, off.cuda(), G, M, 2 * H, C)
    q.qffn_swiglu_quantize_blocks(None, hq, hs, gu, M, H)
    q.qffn_grouped_linear_fp8_blocks(out, hq, hs, q2, s2, off.cuda(), G, M, C, H)
    q.qffn_check_status()
    rr = (x.float() + res.float()).to(bf16).double()
    y = rr / torch.sqrt((rr * rr).mean(1, keepdim=True) + 1e-5) * gain.double()
    y = B.values(*[v.to(torch.float8_e4m3fn).view(u8) if i == 0 else v for i, v in enumerate(B.quantize(y))])
    g_u = B.grouped(y[token], v1, off)[0].to(bf16).double()
    h = g_u[:, :H] / (1 + torch.exp(-g_u[:, :H])) * g_u[:, H:]
    h = B.values(*[v.to(torch.float8_e4m3fn).view(u8) if i == 0 else v for i, v in enumerate(B.quantize(h))])
    assert torch.equal(r.cpu().double(), rr)
    assert _rel(out, B.grouped(h, v2, off)[0]) <= CHAIN


@pytest.mark.parametrize("T,G,top,C,H", [(3, 8, 2, 264, 136), (40, 4, 2, 512, 264), (300, 8, 2, 264, 520), (900, 3, 1, 520, 264)])
def test_experts_training_step(q, T, G, top, C, H):
    """Forward and backward of norm, experts' gate|up, SwiGLU and down in bf16 against autograd in 64 bits."""
    host = dict(x=_t(1, T, C), gain=(torch.randn(C, generator=torch.Generator().manual_seed(3)) * 0.1 + 1).to(bf16),
                w1=_t(4, G, 2 * H, C, std=C ** -0.5), w2=_t(5, G, C, H, std=H ** -0.5))
    token, off = _route(T, G, top, T)
    M = len(token)
    dout = _t(6, M, C, std=0.1)
    d = {k: v.cuda() for k, v in host.items()}
    t, o, do = token.cuda(), off.cuda(), dout.cuda()
    C16 = -(-C // 16) * 16 == C and -(-H // 16) * 16 == H
    y, rstd, gu, h, out = _new(T, C), torch.empty(T, device="cuda"), _new(M, 2 * H), _new(M, H), _new(M, C)
    q.qffn_rmsnorm_absmax(None, y, rstd, None, None, d["x"], d["gain"], 1e-5, T, C)
    rows = y[t]
    q.qffn_grouped_linear(gu, rows, d["w1"], o, G, M, 2 * H, C)
    if C16:
        q.qffn_swiglu_quantize_blocks(h, torch.empty(M, H, dtype=u8, device="cuda"), torch.empty(M, -(-H // 128), dtype=u8, device="cuda"), gu, M, H)
    else:
        q.qffn_swiglu_quant(h, torch.empty(M, H, dtype=u8, device="cuda"), torch.zeros(2, device="cuda"), gu, M, H)
    q.qffn_grouped_linear(out, h, d["w2"], o, G, M, C, H)
    dh, dw2, dgu, drows, dw1 = _new(M, H), _new(G, C, H), _new(M, 2 * H), _new(M, C), _new(G, 2 * H, C)
    q.qffn_grouped_linear_backward(dh, dw2, do, h, d["w2"], o, G, M, C, H, False)
    q.qffn_swiglu_backward(dgu, torch.zeros(2, device="cuda"), dh, gu, M, H)
    q.qffn_grouped_linear_backward(drows, dw1, dgu, rows, d["w1"], o, G, M, 2 * H, C, False)
    dy = torch.zeros(T, C, device="cuda").index_add_(0, t, drows.float()).to(bf16)
    dx, dgain = _new(T, C), torch.empty(C, device="cuda")
    q.qffn_rmsnorm_backward(dx, dgain, None, dy, None, d["x"], rstd, d["gain"], T, C, False,
                            torch.empty(q.qffn_norm_backward_workspace_size(T, C), dtype=u8, device="cuda"))
    q.qffn_check_status()
    lv = {k: v.double().requires_grad_() for k, v in host.items()}
    yy = lv["x"] / torch.sqrt((lv["x"] ** 2).mean(1, keepdim=True) + 1e-5) * lv["gain"]
    yy = yy[token]
    parts = []
    for g, (a, b) in enumerate(B.groups(off, M)):
        z = yy[a:b] @ lv["w1"][g].t()
        parts.append((torch.nn.functional.silu(z[:, :H]) * z[:, H:]) @ lv["w2"][g].t())
    oo = torch.cat(parts)
    oo.backward(dout.double())
    assert _rel(out, oo.detach()) <= CHAIN
    for name, got in (("x", dx), ("gain", dgain), ("w1", dw1), ("w2", dw2)):
        assert _rel(got, lv[name].grad) <= CHAIN, name
