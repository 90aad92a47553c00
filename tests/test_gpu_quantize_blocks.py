"""E4M3 with a scale per block of 128: rows, weights, RMS norm and SwiGLU against the 64-bit plain forms."""
import pytest
import torch

import plain_blocks as B
import plain_ops as P

pytestmark = pytest.mark.gpu
bf16, f32, u8 = torch.bfloat16, torch.float32, torch.uint8
# an fp32 sum of C squares over registers, lanes and warps: at most 4 * 8 + 10 additions one after the other,
# half of that in its root; the root, the quotient and two products: 2 ** -19 holds them all
NORM_REL = 2.0 ** -19


@pytest.fixture(scope="module")
def q():
    import transformer_ffn_block_gb300 as q
    return q


def _t(seed, *shape, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    t = torch.randn(*shape, generator=g) * std + mean
    return (t * torch.exp2(torch.randint(-6, 6, shape[:-1] + (1,), generator=g).float())).to(bf16)


def _codes(rows, cols, by=1, count=None):
    lead = () if count is None else (count,)
    return (torch.full((*lead, rows, cols), 0x55, dtype=u8, device="cuda"),
            torch.full((*lead, -(-rows // by), -(-cols // 128)), 0x55, dtype=u8, device="cuda"))


def _same(got, want_q, want_code):
    """Bit for bit (zeros may have either sign)."""
    v = got[0].cpu().view(torch.float8_e4m3fn).float().double()
    assert torch.equal(got[1].cpu(), want_code)
    assert torch.equal(torch.nan_to_num(v, nan=1e9), torch.nan_to_num(want_q, nan=1e9))


SHAPES = [(1, 16), (1, 128), (3, 144), (5, 240), (7, 1040), (130, 256), (33, 4096), (2, 14336), (257, 112), (1, 1 << 20)]


@pytest.mark.parametrize("rows,cols", SHAPES)
def test_rows(q, rows, cols):
    x = _t(rows + cols, rows, cols)
    x[0, :16] = 0
    if cols > 256:
        x[-1, 128:256] = 0                                          # a block of zeros
        x[0, 130] = 1.75 * 2.0 ** 9                                 # exactly the largest that a scale holds
    d = _codes(rows, cols)
    q.qffn_quantize_blocks(*d, x.cuda(), rows, cols)
    if rows * cols > 1 << 19:                                       # (the plain form goes block by block)
        _same((d[0][:, -4096:], d[1][:, -32:]), *B.quantize(x[:, -4096:].double()))
    else:
        _same(d, *B.quantize(x.double()))


def test_rows_special_values(q):
    x = _t(0, 6, 512)
    x[0, 3] = float("inf")
    x[1, 200] = float("nan")
    x[2, 300] = -float("inf")
    x[3] = 2.0 ** -133                                              # the smallest bf16 values
    x[3, 5] = -(2.0 ** -126)
    x[4] = torch.finfo(bf16).max
    x[5] = 0
    d = _codes(6, 512)
    q.qffn_quantize_blocks(*d, x.cuda(), 6, 512)
    _same(d, *B.quantize(x.double()))
    assert d[1][0].tolist()[0] == 255 and d[1][5].tolist() == [127] * 4 and d[1][3, 1] == 0


def test_every_bf16_magnitude_as_the_largest_of_its_block(q):
    """The scale's rule at each of the 2 ** 15 abs-maxes."""
    bits = torch.arange(1 << 15, dtype=torch.int32).to(torch.int16)
    x = torch.zeros(1 << 15, 16, dtype=torch.int16)
    x[:, 7] = bits
    d = _codes(1 << 15, 16)
    q.qffn_quantize_blocks(*d, x.view(bf16).cuda(), 1 << 15, 16)
    v = x.view(bf16).double()[:, 7]
    c = d[1].cpu()[:, 0].double()
    fin = torch.isfinite(v)
    assert bool((c[~fin] == 255).all()) and c[0] == 127
    v, c = v[fin][1:], c[fin][1:]
    assert bool((v <= 448 * 2.0 ** (c - 127)).all()) and bool(((v > 224 * 2.0 ** (c - 127)) | (c == 0)).all())


@pytest.mark.parametrize("count,rows,cols", [(1, 128, 128), (1, 8, 16), (2, 200, 272), (3, 129, 144), (5, 64, 1024), (1, 1000, 4096)])
def test_weights(q, count, rows, cols):
    w = _t(count + rows, count, rows, cols, std=0.02)
    d = _codes(rows, cols, 128, count)
    q.qffn_quantize_weight_blocks(*d, w.cuda(), count, rows, cols)
    for g in range(count):
        _same((d[0][g], d[1][g]), *B.quantize(w[g].double(), 128))


@pytest.mark.parametrize("N,C", [(1, 16), (1, 4096), (3, 144), (9, 1008), (5, 1040), (130, 2048), (2, 4112), (7, 8192), (3, 16384), (300, 5008)])
@pytest.mark.parametrize("residual", [False, True])
def test_rmsnorm(q, N, C, residual):
    x, gain = _t(N, N, C), (torch.randn(C, generator=torch.Generator().manual_seed(C)) * 0.1 + 1).to(bf16)
    res = _t(N + 7, N, C) if residual else None
    r, y = (torch.full((N, C), float("nan"), dtype=bf16, device="cuda") for _ in range(2))
    rstd, d = torch.full((N,), float("nan"), device="cuda"), _codes(N, C)
    for out_y in (y, None):                                         # with and without y: the same codes
        e = _codes(N, C)
        q.qffn_rmsnorm_quantize_blocks(r if residual else None, out_y, *e, rstd, res.cuda() if residual else None, x.cuda(),
                                       gain.cuda(), 1e-5, N, C)
        if out_y is not None:
            d = e
    assert torch.equal(d[0], e[0]) and torch.equal(d[1], e[1])
    want_r = x if res is None else (x.float() + res.float()).to(bf16)
    if residual:
        assert torch.equal(r.cpu(), want_r)
    v = want_r.double()
    want_rstd = 1 / torch.sqrt((v * v).mean(1) + 1e-5)
    want = v * want_rstd[:, None] * gain.double()
    P.check(rstd, want_rstd, NORM_REL * want_rstd, "rstd")
    P.check(y, want, (P.HALF + 2 * NORM_REL) * want.abs() + 1e-38, "y")
    B.check_blocks(*d, want, 2 * NORM_REL, "codes")


@pytest.mark.parametrize("C", [528, 784, 1296, 2064, 4112, 6144, 6160, 8208, 10240, 10256, 12304, 14336, 14352, 16384])
@pytest.mark.parametrize("few", [False, True])
def test_rmsnorm_of_every_width(q, C, few):
    """Rows on both sides of each number of threads, in calls of few rows and of many."""
    test_rmsnorm(q, 5 if few else 5_100_000 // C, C, True)


def test_rmsnorm_in_place_and_zero_rows(q):
    N, C = 20, 528
    x, res = _t(1, N, C), _t(2, N, C)
    x[4], res[4] = 0, 0
    gain = torch.ones(C, dtype=bf16, device="cuda")
    want = [torch.empty(N, C, dtype=bf16, device="cuda"), *_codes(N, C), torch.empty(N, device="cuda")]
    q.qffn_rmsnorm_quantize_blocks(want[0], None, want[1], want[2], want[3], res.cuda(), x.cuda(), gain, 1e-5, N, C)
    assert want[1][4].eq(0).all() and want[2][4].eq(127).all()
    for alias in (0, 1):                                            # res_out in the place of res_in, of x
        dx, dr, d, rstd = x.cuda(), res.cuda(), _codes(N, C), torch.empty(N, device="cuda")
        q.qffn_rmsnorm_quantize_blocks((dr, dx)[alias], None, *d, rstd, dr, dx, gain, 1e-5, N, C)
        for a, b in zip(((dr, dx)[alias], *d, rstd), want):
            assert torch.equal(a, b)


def test_rmsnorm_of_rows_without_a_number(q):
    """A NaN or an infinity in a row makes that row's blocks NaN and leaves the others alone."""
    N, C = 6, 400
    x = _t(3, N, C)
    clean = x.clone()
    x[2, 17], x[4, 399] = float("nan"), float("inf")
    gain = torch.ones(C, dtype=bf16, device="cuda")
    outs = []
    for t in (x, clean):
        d, rstd = _codes(N, C), torch.empty(N, device="cuda")
        q.qffn_rmsnorm_quantize_blocks(None, None, *d, rstd, None, t.cuda(), gain, 1e-5, N, C)
        outs.append((*d, rstd))
    good = [0, 1, 3, 5]
    for a, b in zip(*outs):
        assert torch.equal(a[good], b[good])
    assert outs[0][1][2].eq(255).all() and outs[0][1][4, 3] == 255


@pytest.mark.parametrize("N,H", [(1, 16), (1, 2048), (3, 144), (37, 2048), (130, 400), (5, 14336), (1000, 272)])
def test_swiglu(q, N, H):
    gu = _t(N + H, N, 2 * H)
    h = torch.full((N, H), float("nan"), dtype=bf16, device="cuda")
    d, e = _codes(N, H), _codes(N, H)
    q.qffn_swiglu_quantize_blocks(h, *d, gu.cuda(), N, H)
    q.qffn_swiglu_quantize_blocks(None, *e, gu.cuda(), N, H)
    assert torch.equal(d[0], e[0]) and torch.equal(d[1], e[1])
    g, u = gu.double()[:, :H], gu.double()[:, H:]
    want = g / (1 + torch.exp(-g)) * u
    # the exponential, its quotient, two products; and a sigmoid below the smallest normal number, 2 ** -126, is flushed to
    # zero (its reciprocal is): off by less than 2 ** -126, which the two products multiply by g and u
    P.check(h, want, (P.HALF + P.ACT_REL) * want.abs() + 2.0 ** -126 * (g * u).abs(), "h")
    B.check_blocks(*d, want, P.ACT_REL, "codes")


def test_rows_past_two_to_the_31(q):
    """Offsets of more than 31 bits: the last rows of a tensor of 2^31 + 2^20 values."""
    rows, cols = (1 << 11) + 1, 1 << 20
    x = torch.zeros(rows, cols, dtype=bf16, device="cuda")
    last = _t(5, 1, cols)
    x[-1] = last[0].cuda()
    d = _codes(rows, cols)
    q.qffn_quantize_blocks(*d, x, rows, cols)
    one = _codes(1, cols)
    q.qffn_quantize_blocks(*one, last.cuda(), 1, cols)
    assert torch.equal(d[0][-1], one[0][0]) and torch.equal(d[1][-1], one[1][0])
    assert not d[0][:-1].any() and bool((d[1][:-1] == 127).all())
