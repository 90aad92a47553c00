"""GPU parity of the layer norm and of the norms' backward against 64-bit plain forms."""
import pytest
import torch

import plain_ops as P
from test_gpu_canaries import Guarded

pytestmark = pytest.mark.gpu

SHAPES = [(1, 8), (3, 64), (77, 264), (20, 512), (5, 1000), (130, 1032), (33, 2048), (700, 4096), (9, 4104), (4, 8192),
          (300, 8200), (3, 16384)]


@pytest.fixture(scope="module")
def q():
    import transformer_ffn_block_gb300 as q
    return q


def _rows(N, C, seed):
    g = torch.Generator().manual_seed(seed)
    t = torch.randn(N, C, generator=g) * torch.rand(N, 1, generator=g).add(0.2)
    if N > 2:
        t[1] = 100.0 + 0.5 * t[1]          # a large common offset
        t[2] = 3.0                         # a constant row: variance zero
    return t.to(torch.bfloat16)


def _vec(C, seed, std=0.2, mean=0.0):
    return (torch.randn(C, generator=torch.Generator().manual_seed(seed)) * std + mean).to(torch.bfloat16)


def _empty(*shape, dtype=torch.bfloat16):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def _check_forward(y, mean, rstd, r, gain, shift, eps):
    r64, g64 = r.double().cpu(), gain.double()
    want, wm, ws = P.layernorm(r64, g64, None if shift is None else shift.double(), eps)
    size = r64.abs().mean(1)
    P.check(mean, wm, 2.0 ** -19 * size, "mean")
    d_mean = 2.0 ** -19 * size
    P.check(rstd, ws, 2.0 ** -18 * ws + ws ** 3 * d_mean ** 2, "rstd")
    hat = (r64 - wm[:, None]) * ws[:, None]
    e = g64.abs() * (ws * d_mean)[:, None] + (2.0 ** -17 + (ws * d_mean)[:, None] ** 2) * (hat * g64).abs()
    P.check(y, want, P.HALF * (want.abs() + e) + e, "y")


@pytest.mark.parametrize("N,C", SHAPES)
@pytest.mark.parametrize("residual,shift", [(False, True), (True, True), (True, False)])
def test_layernorm(q, N, C, residual, shift):
    x, res = _rows(N, C, N + C), (_rows(N, C, 7) if residual else None)
    gain, sh = _vec(C, 1, mean=1.0), (_vec(C, 2) if shift else None)
    y, r = Guarded(N * C * 2), Guarded(N * C * 2)
    mean, rstd = Guarded(N * 4), Guarded(N * 4)
    stats = torch.full((2,), 9.0, device="cuda")
    bf, f32 = torch.bfloat16, torch.float32
    q.qffn_layernorm_absmax(r.view(bf, N, C) if residual else None, y.view(bf, N, C), mean.view(f32, N), rstd.view(f32, N),
                            stats, res.cuda() if residual else None, x.cuda(), gain.cuda(), sh.cuda() if shift else None,
                            1e-5, N, C)
    for buf, name in ((y, "y"), (mean, "mean"), (rstd, "rstd")):
        buf.check(name)
    rr = x
    if residual:
        r.check("res_out")
        rr = r.view(bf, N, C).cpu()
        assert torch.equal(rr, x + res)        # a bf16 sum: one rounding
    _check_forward(y.view(bf, N, C), mean.view(f32, N), rstd.view(f32, N), rr, gain, sh, 1e-5)
    assert stats[0].item() == y.view(bf, N, C).float().abs().max().item() and stats[1].item() == 9.0


def test_layernorm_in_place_and_no_stats(q):
    N, C = 37, 4096
    x, res, gain = _rows(N, C, 1).cuda(), _rows(N, C, 2).cuda(), _vec(C, 3, mean=1.0).cuda()
    want, y, y2, m, s = _empty(N, C), _empty(N, C), _empty(N, C), _empty(N, dtype=torch.float32), _empty(N, dtype=torch.float32)
    q.qffn_layernorm_absmax(want, y, m, s, None, res, x, gain, None, 1e-6, N, C)
    for alias in (x, res):
        keep = alias.clone()
        q.qffn_layernorm_absmax(alias, y2, m, s, None, res, x, gain, None, 1e-6, N, C)
        assert torch.equal(alias, want) and torch.equal(y2, y)
        alias.copy_(keep)


def test_layernorm_rows_do_not_mix(q):
    """A row of NaN or infinities stays its own: the others are what they are without it."""
    N, C = 6, 264
    x = _rows(N, C, 5)
    bad = x.clone()
    bad[3] = float("nan")
    bad[4, 10] = float("inf")
    gain = _vec(C, 3, mean=1.0).cuda()
    out = []
    for t in (x, bad):
        y, m, s = _empty(N, C), _empty(N, dtype=torch.float32), _empty(N, dtype=torch.float32)
        q.qffn_layernorm_absmax(None, y, m, s, None, None, t.cuda(), gain, None, 1e-5, N, C)
        out.append(y.cpu())
    keep = [0, 1, 2, 5]
    assert torch.equal(out[0][keep], out[1][keep])
    assert out[1][3].isnan().all() and out[1][4].isnan().any()


@pytest.mark.parametrize("N,C", SHAPES)
@pytest.mark.parametrize("rms", [False, True])
@pytest.mark.parametrize("dres,accumulate", [(True, False), (False, True)])
def test_norm_backward(q, N, C, rms, dres, accumulate):
    g = torch.Generator().manual_seed(N * 3 + C)
    r, gain = _rows(N, C, N + 2 * C), _vec(C, 4, mean=1.0)
    dy = (torch.randn(N, C, generator=g) * 0.1).to(torch.bfloat16)
    dr = (torch.randn(N, C, generator=g) * 0.1).to(torch.bfloat16) if dres else None
    mean = None if rms else r.float().mean(1)
    mid = r.float() - (0 if rms else mean[:, None])
    rstd = (mid.square().mean(1) + 1e-5).rsqrt()
    old = torch.randn(2, C, generator=g)
    dx, dg, ds = Guarded(N * C * 2), Guarded(C * 4), Guarded(C * 4)
    bf, f32 = torch.bfloat16, torch.float32
    dgv, dsv, dxv = dg.view(f32, C), ds.view(f32, C), dx.view(bf, N, C)
    dgv.copy_(old[0]), dsv.copy_(old[1])
    size = q.qffn_norm_backward_workspace_size(N, C)
    ws = Guarded(size)
    stats = torch.full((2,), 9.0, device="cuda")
    drc = dr.cuda() if dres else None
    if rms:
        q.qffn_rmsnorm_backward(dxv, dgv, stats, dy.cuda(), drc, r.cuda(), rstd.cuda(), gain.cuda(), N, C, accumulate,
                                ws.view(torch.uint8, size))
    else:
        q.qffn_layernorm_backward(dxv, dgv, dsv, stats, dy.cuda(), drc, r.cuda(), mean.cuda(), rstd.cuda(), gain.cuda(),
                                  N, C, accumulate, ws.view(torch.uint8, size))
    for buf, name in ((dx, "dx"), (dg, "dgain"), (ds, "dshift"), (ws, "workspace")):
        buf.check(name)
    wdx, wdg, wds, b_dx, b_dg, b_ds = P.norm_backward(dy.double(), dr.double() if dres else None, r.double(),
                                                      None if rms else mean.double(), rstd.double(), gain.double())
    add = old.double() if accumulate else torch.zeros(2, C, dtype=torch.float64)
    P.check(dxv, wdx, b_dx, "dx")
    P.check(dgv, wdg + add[0], b_dg + 2.0 ** -23 * (wdg.abs() + add[0].abs()), "dgain")
    if not rms:
        P.check(dsv, wds + add[1], b_ds + 2.0 ** -23 * (wds.abs() + add[1].abs()), "dshift")
    assert stats[0].item() == dxv.float().abs().max().item() and stats[1].item() == 9.0


def test_norm_backward_same_bits_in_place_and_without_dshift(q):
    N, C = 1234, 4096
    g = torch.Generator().manual_seed(3)
    r, gain = _rows(N, C, 9).cuda(), _vec(C, 4, mean=1.0).cuda()
    dy = (torch.randn(N, C, generator=g) * 0.1).to(torch.bfloat16).cuda()
    dr = (torch.randn(N, C, generator=g) * 0.1).to(torch.bfloat16).cuda()
    mean = r.float().mean(1)
    rstd = (r.float().var(1, correction=0) + 1e-5).rsqrt()
    ws = torch.empty(q.qffn_norm_backward_workspace_size(N, C), dtype=torch.uint8, device="cuda")

    def run(dx, dyt, drt, dshift=True):
        dg, ds = _empty(C, dtype=torch.float32), _empty(C, dtype=torch.float32)
        q.qffn_layernorm_backward(dx, dg, ds if dshift else None, None, dyt, drt, r, mean, rstd, gain, N, C, False, ws)
        return dx.clone(), dg, ds

    first = run(_empty(N, C), dy, dr)
    for again in (run(_empty(N, C), dy, dr), run(d2 := dy.clone(), d2, dr), run(d3 := dr.clone(), dy, d3)):
        assert all(torch.equal(a, b) for a, b in zip(first, again))
    no_shift = run(_empty(N, C), dy, dr, dshift=False)
    assert torch.equal(first[0], no_shift[0]) and torch.equal(first[1], no_shift[1]) and no_shift[2].isnan().all()


def test_norms_of_no_rows(q):
    C = 64
    gain = _vec(C, 1).cuda()
    none = torch.empty(0, C, dtype=torch.bfloat16, device="cuda")
    p = gain.data_ptr()                   # an address of the device: nothing is read or written through it
    f = torch.empty(1, dtype=torch.float32, device="cuda")
    stats = torch.full((2,), 9.0, device="cuda")
    q.qffn_layernorm_absmax(None, p, f, f, stats, None, p, gain, None, 1e-5, 0, C)
    assert stats.tolist() == [0.0, 9.0]
    ws = torch.empty(q.qffn_norm_backward_workspace_size(0, C), dtype=torch.uint8, device="cuda")
    dg, ds = torch.full((C,), 2.0, device="cuda"), torch.full((C,), 3.0, device="cuda")
    q.qffn_layernorm_backward(p, dg, ds, None, p, None, p, f, f, gain, 0, C, True, ws)
    assert (dg == 2.0).all() and (ds == 3.0).all()
    q.qffn_layernorm_backward(p, dg, ds, None, p, None, p, f, f, gain, 0, C, False, ws)
    assert (dg == 0.0).all() and (ds == 0.0).all() and none.numel() == 0
