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
