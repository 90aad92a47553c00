"""Block-scaled E4M3 and grouped products where a call meets its limits: special values, sizes, calls without rows, bytes
around the outputs, and inputs written by the kernels just before."""
import pytest
import torch

import plain_blocks as B
from test_gpu_canaries import Guarded
from test_gpu_grouped import _new, _t, _wide
from test_gpu_quantize_blocks import _codes, _same

pytestmark = pytest.mark.gpu
bf16, f32, u8, i32 = torch.bfloat16, torch.float32, torch.uint8, torch.int32


@pytest.fixture(scope="module")
def q():
    import transformer_ffn_block_gb300 as q
    return q


# ------------------------------------------------------------------ weights

def test_weights_special_values(q):
    """An infinity or a NaN anywhere in a 128 x 128 makes that block NaN, a block of zeros gets 127, others are theirs."""
    w = _wide(1, 3, 300, 400)
    clean = w.clone()
    w[0, 5, 7], w[1, 200, 300], w[2, 299, 399], w[1, 127, 128] = float("inf"), float("nan"), -float("inf"), float("nan")
    w[0, :128, 128:256] = 0
    w[2, 128:256, :128] = 0
    w[2, 130, 17] = 2.0 ** -133
    got, base = _codes(300, 400, 128, 3), _codes(300, 400, 128, 3)
    q.qffn_quantize_weight_blocks(*got, w.cuda(), 3, 300, 400)
    q.qffn_quantize_weight_blocks(*base, clean.cuda(), 3, 300, 400)
    for g in range(3):
        _same((got[0][g], got[1][g]), *B.quantize(w[g].double(), 128))
    changed = torch.zeros(3, 3, 4, dtype=torch.bool)
    for at in ((0, 0, 0), (1, 1, 2), (2, 2, 3), (1, 0, 1), (0, 0, 1), (2, 1, 0)):
        changed[at] = True
    same = (got[1] == base[1]).cpu()
    assert bool(same[~changed].all())
    assert got[1][0, 0, 0] == 255 and got[1][1, 1, 2] == 255 and got[1][2, 2, 3] == 255 and got[1][0, 0, 1] == 127 and got[1][2, 1, 0] == 0


def test_most_matrices(q):
    """4096 matrices of two row blocks and two columns of blocks each, all different."""
    n, rows, cols = 4096, 136, 144
    w = _wide(2, n, rows, cols)
    d = _codes(rows, cols, 128, n)
    q.qffn_quantize_weight_blocks(*d, w.cuda(), n, rows, cols)
    for g in (0, 1, 2047, 4094, 4095):
        _same((d[0][g], d[1][g]), *B.quantize(w[g].double(), 128))
    # the scale's rule for every block
    pad = torch.nn.functional.pad(w.double(), (0, 256 - cols, 0, 256 - rows)).view(n, 2, 128, 2, 128)
    top, s = pad.abs().amax((2, 4)), torch.exp2(d[1].cpu().double() - 127)
    assert bool((top <= 448 * s).all()) and bool((top > 224 * s).all())


def test_tall_weights(q):
    """More rows of blocks than a launch has in its second dimension."""
    whole, extra = 65535 * 128, 200
    rows, cols = whole + extra, 16
    w = torch.zeros(rows, cols, dtype=bf16, device="cuda")
    first, last = _wide(3, 256, cols), _wide(4, extra, cols) * 3
    w[:256], w[whole:] = first.cuda(), last.cuda()
    d = _codes(rows, cols, 128, 1)
    q.qffn_quantize_weight_blocks(*d, w, 1, rows, cols)
    for part, a, b in ((first, 0, 256), (last, whole, rows)):
        _same((d[0][0, a:b], d[1][0, a // 128:-(-b // 128)]), *B.quantize(part.double(), 128))
    assert not d[0][0, 256:whole].any() and bool((d[1][0, 2:65535] == 127).all())


def test_weights_past_two_to_the_31(q):
    n, rows, cols = 3, 1 << 15, (1 << 15) + 16
    w = torch.zeros(n, rows, cols, dtype=bf16, device="cuda")
    w[-1].normal_(0.0, 0.02, generator=torch.Generator(device="cuda").manual_seed(1))
    w[-1, :, -16:] *= 8.0
    d, one = _codes(rows, cols, 128, n), _codes(rows, cols, 128, 1)
    q.qffn_quantize_weight_blocks(*d, w, n, rows, cols)
    q.qffn_quantize_weight_blocks(*one, w[-1].clone(), 1, rows, cols)
    assert torch.equal(d[0][-1], one[0][0]) and torch.equal(d[1][-1], one[1][0])
    assert not d[0][:-1].any() and bool((d[1][:-1] == 127).all())
    part = w[-1, -256:, -272:].cpu().double()                       # (the last three columns of blocks, the last of 16)
    _same((d[0][-1, -256:, -272:], d[1][-1, -2:, -3:]), *B.quantize(part, 128))


# ------------------------------------------------------------------ SwiGLU

def test_swiglu_special_values(q):
    """A block with a value that is not finite gets 255 and NaN codes; the others are what they were."""
    N, H = 9, 400
    gu = _t(5, N, 2 * H)
    clean = gu.clone()
    inf, nan = float("inf"), float("nan")
    for row, col, g, u in ((0, 3, inf, 1.0), (1, 130, -inf, 1.0), (2, 399, nan, 1.0), (3, 128, 1.0, nan), (4, 255, 1.0, -inf), (5, 256, 0.0, inf),
                           (6, 384, -inf, inf), (7, 17, -3e38, 1.0)):
        gu[row, col], gu[row, H + col] = g, u
    outs = []
    for t in (gu, clean):
        d, h = _codes(N, H), _new(N, H)
        q.qffn_swiglu_quantize_blocks(h, *d, t.cuda(), N, H)
        outs.append((*d, h))
    g, u = gu.double()[:, :H], gu.double()[:, H:]
    want = g / (1 + torch.exp(-g)) * u
    assert torch.equal(torch.isnan(outs[0][2].cpu()), torch.isnan(want))
    codes, base = outs[0][0].cpu(), outs[1][0].cpu()
    for row in range(N):
        for j, (a, b) in enumerate(B.cuts(H)):
            finite = bool(torch.isfinite(want[row, a:b]).all())
            assert (outs[0][1][row, j] == 255) == (not finite), (row, j)
            if not finite:
                assert bool(((codes[row, a:b] & 0x7F) == 0x7F).all())
            elif torch.equal(gu[row, [*range(a, b)]], clean[row, [*range(a, b)]]):
                assert torch.equal(codes[row, a:b], base[row, a:b]) and outs[0][1][row, j] == outs[1][1][row, j]
    assert outs[0][2][7, 17] == 0                                   # silu of a very low number


# ------------------------------------------------------------------ calls without rows

def test_weight_gradients_without_rows(q):
    """No rows at all: dw is cleared, or kept where it is added to."""
    G, N, K = 3, 200, 72
    w, off = _t(1, G, N, K).cuda(), torch.zeros(G + 1, dtype=i32, device="cuda")
    empty = torch.empty(0, N, dtype=bf16, device="cuda"), torch.empty(0, K, dtype=bf16, device="cuda")
    dx = torch.empty(0, K, dtype=bf16, device="cuda")
    guard = Guarded(G * N * K * 2)
    dw = guard.view(bf16, G, N, K)
    old = dw.clone()
    q.qffn_grouped_linear_backward(dx, dw, *empty, w, off, G, 0, N, K, True)
    assert torch.equal(dw.view(torch.int16), old.view(torch.int16))
    q.qffn_grouped_linear_backward(dx, dw, *empty, w, off, G, 0, N, K, False)
    q.qffn_check_status()
    assert not dw.any()
    guard.check("dw")


# ------------------------------------------------------------------ bytes around the outputs

@pytest.mark.parametrize("rows,cols", [(1, 16), (3, 144), (37, 272), (130, 1040), (9, 4112)])
def test_quantisers_stay_inside_their_outputs(q, rows, cols):
    blocks = -(-cols // 128)
    x, gain = _t(1, rows, cols).cuda(), torch.ones(cols, dtype=bf16, device="cuda")
    codes, scale = Guarded(rows * cols), Guarded(rows * blocks)
    q.qffn_quantize_blocks(codes.view(u8, rows, cols), scale.view(u8, rows, blocks), x, rows, cols)
    codes.check("q"), scale.check("scale")
    codes, scale, h = Guarded(rows * cols), Guarded(rows * blocks), Guarded(rows * cols * 2)
    q.qffn_swiglu_quantize_blocks(h.view(bf16, rows, cols), codes.view(u8, rows, cols), scale.view(u8, rows, blocks),
                                  _t(2, rows, 2 * cols).cuda(), rows, cols)
    codes.check("q"), scale.check("scale"), h.check("h")
    r, y, rstd = Guarded(rows * cols * 2), Guarded(rows * cols * 2), Guarded(rows * 4)
    codes, scale = Guarded(rows * cols), Guarded(rows * blocks)
    q.qffn_rmsnorm_quantize_blocks(r.view(bf16, rows, cols), y.view(bf16, rows, cols), codes.view(u8, rows, cols),
                                   scale.view(u8, rows, blocks), rstd.view(f32, rows), x, x, gain, 1e-5, rows, cols)
    codes.check("q"), scale.check("scale"), r.check("res_out"), y.check("y"), rstd.check("rstd")
    brows = -(-rows // 128)
    codes, scale = Guarded(2 * rows * cols), Guarded(2 * brows * blocks)
    q.qffn_quantize_weight_blocks(codes.view(u8, 2, rows, cols), scale.view(u8, 2, brows, blocks), _t(3, 2, rows, cols).cuda(), 2, rows, cols)
    codes.check("q"), scale.check("scale")


@pytest.mark.parametrize("G,M,N,K", [(1, 3, 8, 16), (3, 40, 136, 272), (2, 84, 1008, 3584), (4, 700, 1032, 400), (2, 1235, 2376, 528), (4, 40, 8200, 208)])
def test_products_stay_inside_their_outputs(q, G, M, N, K):
    x, w, dout = _t(1, M, K).cuda(), _t(2, G, N, K, std=0.1).cuda(), _t(3, M, N).cuda()
    off = torch.linspace(0, M, G + 1).to(i32).cuda()
    xr, wr = _codes(M, K), _codes(N, K, 128, G)
    q.qffn_quantize_blocks(*xr, x, M, K)
    q.qffn_quantize_weight_blocks(*wr, w, G, N, K)
    for call in (lambda o: q.qffn_grouped_linear(o, x, w, off, G, M, N, K),
                 lambda o: q.qffn_grouped_linear_fp8_blocks(o, *xr, *wr, off, G, M, N, K),
                 lambda o: q.qffn_linear_fp8_blocks(o, *xr, wr[0][0], wr[1][0], None, o, M, N, K)):
        out = Guarded(M * N * 2)
        call(out.view(bf16, M, N))
        out.check("out")
    for accumulate in (False, True):
        dx, dw = Guarded(M * K * 2), Guarded(G * N * K * 2)
        q.qffn_grouped_linear_backward(dx.view(bf16, M, K), dw.view(bf16, G, N, K), dout, x, w, off, G, M, N, K, accumulate)
        dx.check("dx"), dw.check("dw")
    q.qffn_check_status()


# ------------------------------------------------------------------ gradients of long rows (two kernels side by side)

@pytest.mark.parametrize("M", [6, 40])
def test_gradients_of_long_rows_do_not_mix(q, M):
    """What a neighbour, an empty group's matrix or a row of no group holds reaches no other gradient."""
    G, N, K = 4, 8200, 208
    off = torch.tensor([1, M // 4 + 1, M // 2, M // 2, M - 1], dtype=i32)
    dout, x, w = _t(1, M, N), _t(2, M, K), _t(3, G, N, K)
    bad = slice(int(off[1]), int(off[2]))

    def run():
        dx, dw = _new(M, K), _new(G, N, K)
        q.qffn_grouped_linear_backward(dx, dw, dout.cuda(), x.cuda(), w.cuda(), off.cuda(), G, M, N, K, False)
        q.qffn_check_status()
        return dx, dw

    base_dx, base_dw = run()
    live = torch.zeros(M, dtype=torch.bool)
    live[1:M - 1] = True
    assert torch.equal(torch.isfinite(base_dx).all(1).cpu(), live) and torch.isfinite(base_dw).all()
    dout[bad], w[1] = float("nan"), float("inf")
    for t in (x, dout):
        t[0], t[-1] = float("inf"), float("nan")
    x[bad], w[2] = float("-inf"), float("nan")
    dx, dw = run()
    base_dx[bad], base_dw[1] = float("nan"), float("nan")
    for got, want in ((dx, base_dx), (dw, base_dw)):
        assert torch.equal(torch.nan_to_num(got, nan=7.0), torch.nan_to_num(want, nan=7.0))
    assert not dw[2].any()


@pytest.mark.parametrize("M", [3, 40])
@pytest.mark.parametrize("graph", [False, True])
def test_gradients_of_long_rows_on_the_results_of_the_calls_before(q, M, graph):
    """x, dout, the matrices and the previous gradient written by kernels that let the next one start before they have
    written, the last rows last, in front of the two kernels of the gradients: the bits of the same calls with a
    synchronisation behind each."""
    G, N, K, big, rounds = 4, 8208, 208, 3000, 6
    off = torch.tensor([0, M // 3, M // 3, M - 1, M], dtype=i32, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(M)

    def rand(*s, std=1.0):
        return torch.empty(*s, device="cuda").normal_(0.0, std, generator=gen).to(bf16)

    inputs = [(rand(big, 2 * N), rand(M, K), rand(G * N, K, std=0.1)) for _ in range(rounds)]
    gain = torch.ones(K, dtype=bf16, device="cuda")
    h, x, w = (torch.zeros(*s, dtype=bf16, device="cuda") for s in ((big, N), (M, K), (G * N, K)))
    dout = h[big - M:]
    codes, scale = torch.empty(big * N, dtype=u8, device="cuda"), torch.empty(max(big * 65, G * N * 2), dtype=u8, device="cuda")
    rstd = torch.empty(G * N, device="cuda")
    results = [(_new(M, K), _new(G, N, K), _new(M, K)) for _ in range(rounds)]

    def run(step):
        for (gu, xs, ws), (dx, dw, dx2) in zip(inputs, results):
            q.qffn_rmsnorm_quantize_blocks(None, w, codes, scale, rstd, None, ws, gain, 1e-5, G * N, K)
            step()
            q.qffn_rmsnorm_quantize_blocks(None, x, codes, scale, rstd, None, xs, gain, 1e-5, M, K)
            step()
            q.qffn_swiglu_quantize_blocks(h, codes, scale, gu, big, N)
            step()
            q.qffn_grouped_linear_backward(dx, dw, dout, x, w, off, G, M, N, K, False)
            step()
            q.qffn_grouped_linear_backward(dx2, dw, dout, x, w, off, G, M, N, K, True)     # (onto the gradient just written)
            step()

    run(torch.cuda.synchronize)
    want = [tuple(t.clone() for t in r) for r in results]
    assert all(torch.isfinite(t).all() for r in want for t in r)
    for r in results:
        for t in r:
            t.fill_(float("nan"))
    if graph:
        torch.cuda.synchronize()
        captured = torch.cuda.CUDAGraph()
        with torch.cuda.graph(captured):
            run(lambda: None)
    for _ in range(4):
        if graph:
            captured.replay()
        else:
            run(lambda: None)
        q.qffn_check_status()
        for a, b in zip(results, want):
            assert all(torch.equal(s, t) for s, t in zip(a, b))
