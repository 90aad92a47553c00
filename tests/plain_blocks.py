"""Plain 64-bit forms of the block-scaled E4M3 operators and the products grouped by expert (torch float64 on
the CPU), and the error bounds their kernels are held to."""
import torch

from plain_ops import ACC, HALF

HALF_E4M3 = 2.0 ** -4        # half an E4M3 step, relative to the value
TINY_E4M3 = 2.0 ** -10       # half of E4M3's smallest step, relative to the scale


def cuts(n):
    return [(a, min(a + 128, n)) for a in range(0, n, 128)]


def code_of(amax):
    """E8M0 code of one abs-max (a Python float), by trying the powers of two."""
    if amax != amax or amax in (float("inf"),):
        return 255
    if amax == 0:
        return 127
    c = 0
    while amax > 448 * 2.0 ** (c - 127):
        c += 1
    return c


def e4m3(v):
    """v (float64) rounded to E4M3, nearest even, saturating."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -30))).clamp_min(-6)
    e = torch.where(v.abs() >= 2.0 ** (e + 1), e + 1, e)          # (log2 is rounded)
    e = torch.where(v.abs() < 2.0 ** e, (e - 1).clamp_min(-6), e)
    step = 2.0 ** (e - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def quantize(v, by=1):
    """Values (unscaled codes) and scale codes of v [rows, cols]; blocks of ``by`` rows x 128 columns."""
    rows, cols = v.shape
    q = torch.zeros_like(v)
    rcuts = [(a, min(a + by, rows)) for a in range(0, rows, by)]
    code = torch.zeros(len(rcuts), len(cuts(cols)), dtype=torch.uint8)
    for i, (r0, r1) in enumerate(rcuts):
        for j, (c0, c1) in enumerate(cuts(cols)):
            b = v[r0:r1, c0:c1]
            c = code_of(float("nan") if not torch.isfinite(b).all() else b.abs().max().item())
            code[i, j] = c
            q[r0:r1, c0:c1] = float("nan") if c == 255 else e4m3(b * 2.0 ** (127 - c))
    return q, code


def scales(code):
    return torch.where(code == 255, torch.full(code.shape, float("nan"), dtype=torch.float64), 2.0 ** (code.double() - 127))


def values(q, code, by=1):
    """What codes (uint8 or float8) stand for."""
    v = q.view(torch.float8_e4m3fn).float().double()
    s = scales(code.view(torch.uint8)).repeat_interleave(128, 1)[:, :v.shape[1]]
    return v * (s.repeat_interleave(by, 0)[:v.shape[0]] if by > 1 else s)


def check_blocks(q, code, want, rel, name):
    """Codes and scales of values that are ``want`` to the relative error ``rel``: the scale is the smallest power of two
    that holds the block (within rel), and each code the nearest (within rel)."""
    q, code = q.cpu(), code.cpu().view(torch.uint8)
    got = values(q, code)
    s = scales(code)
    for j, (a, b) in enumerate(cuts(want.shape[1])):
        top = want[:, a:b].abs().amax(1)
        assert bool((top * (1 - rel) <= 448 * s[:, j]).all()), name
        assert bool(((top * (1 + rel) > 224 * s[:, j]) | (code[:, j] == 0) | ((top == 0) & (code[:, j] == 127))).all()), name
    full = s.repeat_interleave(128, 1)[:, :want.shape[1]]
    bound = torch.maximum(HALF_E4M3 * want.abs(), TINY_E4M3 * full) * (1 + 2 * rel) + rel * want.abs()
    err = (got - want).abs()
    assert bool((err <= bound).all()), (name, float((err / bound.clamp_min(1e-300)).max()))


def linear(x, w, bias=None, residual=None):
    """x [M,K] and w [N,K] as the values that the operands stand for; out and its bound."""
    out = x @ w.t()
    e = (x.shape[1] * ACC + 2.0 ** -21) * (x.abs() @ w.abs().t())
    for t in (bias, residual):
        if t is not None:
            out = out + t
            e = e + 2.0 ** -23 * (out.abs() + t.abs())
    return out, HALF * (out.abs() + e) + e


def groups(offsets, M):
    """(first row, end) of each group, as the calls read the offsets."""
    o = [0]
    for v in offsets:
        o.append(max(o[-1], min(max(int(v), 0), M)))
    return list(zip(o[1:-1], o[2:]))


def grouped(x, w, offsets):
    """w [G,N,K] values; out [M,N], its bound, and which rows are written."""
    M, N = x.shape[0], w.shape[1]
    out, bound = torch.zeros(M, N, dtype=torch.float64), torch.zeros(M, N, dtype=torch.float64)
    live = torch.zeros(M, dtype=torch.bool)
    for g, (a, b) in enumerate(groups(offsets, M)):
        if b > a:
            out[a:b], bound[a:b] = linear(x[a:b], w[g])
            live[a:b] = True
    return out, bound, live


def grouped_backward(dout, x, w, offsets, old=None):
    """dx, dw, their bounds, and which rows of dx are written."""
    G, N, K = w.shape
    dx, b_dx = torch.zeros_like(x), torch.zeros_like(x)
    dw, b_dw = torch.zeros_like(w), torch.zeros_like(w)
    live = torch.zeros(x.shape[0], dtype=torch.bool)
    for g, (a, b) in enumerate(groups(offsets, x.shape[0])):
        if b > a:
            dx[a:b], b_dx[a:b] = linear(dout[a:b], w[g].t())
            live[a:b] = True
        d, t = dout[a:b], x[a:b]
        dw[g] = d.t() @ t
        e = ((b - a) * ACC + 2.0 ** -21) * (d.abs().t() @ t.abs())
        if old is not None:
            dw[g] = dw[g] + old[g]
            e = e + 2.0 ** -23 * (dw[g].abs() + old[g].abs())
        b_dw[g] = HALF * (dw[g].abs() + e) + e
    return dx, dw, b_dx, b_dw, live
