"""Calls that start on an idle GPU, and calls whose every input was just written, give the bits of the 64-bit forms' tests
again and again, whichever warp of a kernel is first."""
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


def _on_device(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(*shape, device="cuda").normal_(0.0, std, generator=g).to(bf16)


def _records(q, x, by):
    lead, (rows, cols) = x.shape[:-2], x.shape[-2:]
    c = torch.empty(*lead, rows, cols, dtype=u8, device="cuda")
    s = torch.empty(*lead, -(-rows // by), -(-cols // 128), dtype=u8, device="cuda")
    if by == 1:
        q.qffn_quantize_blocks(c, s, x, rows, cols)
    else:
        q.qffn_quantize_weight_blocks(c, s, x, x.shape[0], rows, cols)
    return c, s


def _new(*shape):
    return torch.full(shape, float("nan"), dtype=bf16, device="cuda")


@pytest.mark.parametrize("G", [1, 2, 40])
@pytest.mark.parametrize("form", ["bf16", "E4M3", "backward", "dw"])
def test_calls_on_an_idle_gpu(q, form, G):
    """The groups' table is made while nothing precedes the kernel, so as early as it can be."""
    M, N, K = 1235, 2376, 528
    x, w, d = _on_device(1, M, K), _on_device(2, G, N, K, std=0.1), _on_device(3, M, N, std=0.1)
    off = torch.linspace(0, M, G + 1).to(torch.int32)
    o = off.cuda()
    out, dx, dw = _new(M, N), _new(M, K), _new(G, N, K)
    if form == "E4M3":
        xr, wr = _records(q, x, 1), _records(q, w, 128)
        xv = B.values(*(t.cpu() for t in xr))
        wv = torch.stack([B.values(wr[0][g].cpu(), wr[1][g].cpu(), 128) for g in range(G)])
    else:
        xv, wv = x.cpu().double(), w.cpu().double()

    def call():
        if form == "E4M3":
            q.qffn_grouped_linear_fp8_blocks(out, *xr, *wr, o, G, M, N, K)
        elif form == "bf16":
            q.qffn_grouped_linear(out, x, w, o, G, M, N, K)
        else:
            q.qffn_grouped_linear_backward(dx if form == "backward" else None, dw, d, x, w, o, G, M, N, K, False)

    def results():
        return (out,) if form in ("bf16", "E4M3") else (dx, dw) if form == "backward" else (dw,)

    first = None
    for _ in range(30):
        for t in results():
            t.fill_(float("nan"))
        torch.cuda.synchronize()
        call()
        q.qffn_check_status()                                       # (waits for the call, and raises where a wait ran out)
        first = first or [t.clone() for t in results()]
        assert all(torch.equal(a, b) for a, b in zip(first, results()))
    if form in ("bf16", "E4M3"):
        want, bound, _ = B.grouped(xv, wv, off)
        P.check(first[0], want, bound, "out")
    else:
        want_dx, want_dw, b_dx, b_dw, _ = B.grouped_backward(d.cpu().double(), xv, wv, off)
        if form == "backward":
            P.check(first[0], want_dx, b_dx, "dx")
        P.check(first[-1], want_dw, b_dw, "dw")


def _whole(gen, *shape):
    """Whole numbers of -2 .. 2, whose products sum exactly in 32 bits in any order."""
    return torch.randint(-2, 3, shape, generator=gen, device="cuda")


def test_scales_of_every_call(q):
    """Codes and scales written anew for each call, sums exact: each product is multiplied by its own call's scales."""
    G, M, N, K = 3, 1500, 2376, 1200
    gen = torch.Generator(device="cuda").manual_seed(1)
    blocks, rows = -(-K // 128), -(-N // 128)
    x, xs = torch.empty(M, K, dtype=u8, device="cuda"), torch.empty(M, blocks, dtype=u8, device="cuda")
    w, ws = torch.empty(G, N, K, dtype=u8, device="cuda"), torch.empty(G, rows, blocks, dtype=u8, device="cuda")
    off = torch.empty(G + 1, dtype=torch.int32, device="cuda")
    calls = []
    for i in range(24):
        v, u = _whole(gen, M, K).float(), _whole(gen, G, N, K).float()
        vs, us = (torch.randint(125, 130, s, generator=gen, device="cuda") for s in ((M, blocks), (G, rows, blocks)))
        ends = [0, 1 + (37 * i) % 700, 701 + (53 * i) % 600, M]
        calls.append((v.to(torch.float8_e4m3fn).view(u8), vs.to(u8), u.to(torch.float8_e4m3fn).view(u8), us.to(u8),
                      torch.tensor(ends, dtype=torch.int32, device="cuda")))
    torch.cuda.synchronize()
    outs = []
    for c in calls:
        for dst, src in zip((x, xs, w, ws, off), c):
            dst.copy_(src)
        out = _new(M, N)
        q.qffn_grouped_linear_fp8_blocks(out, x, xs, w, ws, off, G, M, N, K)
        outs.append(out)
    q.qffn_check_status()
    for out, (v, vs, u, us, ends) in zip(outs, calls):
        xv = v.view(torch.float8_e4m3fn).double() * torch.exp2(vs.double() - 127).repeat_interleave(128, 1)[:, :K]
        for g in range(G):
            a, b = int(ends[g]), int(ends[g + 1])
            scale = torch.exp2(us[g].double() - 127).repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)[:, :K]
            want = xv[a:b] @ (u[g].view(torch.float8_e4m3fn).double() * scale).t()
            # (|sum| < 2^22 units of 2^-4 at most: exact in 32 bits, then rounded once)
            assert torch.equal(out[a:b], want.float().to(bf16))


@pytest.mark.parametrize("N,K", [(264, 200), (72, 520), (320, 328)])
@pytest.mark.parametrize("spare", [0, 1, 40])
def test_weight_gradients_of_groups_of_every_length(q, N, K, spare):
    """Groups of 1 to 130 rows, so ending at each row of a stage, in another order each call; sums exact.  Rows of no group
    hold NaN, the neighbours' others."""
    gen = torch.Generator(device="cuda").manual_seed(N + spare)
    host = torch.Generator().manual_seed(N + spare)
    G = 130
    used = G * (G + 1) // 2
    M = used + spare
    dout, x = torch.empty(M, N, dtype=bf16, device="cuda"), torch.empty(M, K, dtype=bf16, device="cuda")
    w, off = torch.zeros(G, N, K, dtype=bf16, device="cuda"), torch.empty(G + 1, dtype=torch.int32, device="cuda")
    for _ in range(6):
        sizes = torch.randperm(G, generator=host) + 1
        ends = torch.cat([torch.zeros(1, dtype=torch.long), sizes.cumsum(0)])
        d, v = _whole(gen, M, N).to(bf16), _whole(gen, M, K).to(bf16)
        d[used:], v[used:] = float("nan"), float("nan")
        old = _whole(gen, G, N, K).to(bf16)
        results = []
        for accumulate in (False, True):
            dw = old.clone() if accumulate else _new(G, N, K)
            dout.copy_(d)
            x.copy_(v)
            off.copy_(ends)
            q.qffn_grouped_linear_backward(None, dw, dout, x, w, off, G, M, N, K, accumulate)
            results.append(dw)
        q.qffn_check_status()
        for g in range(G):
            a, b = int(ends[g]), int(ends[g + 1])
            want = d[a:b].double().t() @ v[a:b].double()
            assert torch.equal(results[0][g], want.float().to(bf16)), g
            assert torch.equal(results[1][g], (want + old[g].double()).float().to(bf16)), g
