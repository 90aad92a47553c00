"""The layer norm's backward on rows far from zero: xhat = (r - mean) * rstd to the rounding of the difference and
of the product, whatever the mean."""
import pytest
import torch

import plain_ops as P

pytestmark = pytest.mark.gpu
bf16, f32 = torch.bfloat16, torch.float32

# a warp per row, one launch for few rows, the ring of each width
SHAPES = [(40, 264), (700, 264), (1, 4096), (77, 2048), (300, 4096), (700, 4096), (600, 1000), (515, 8200), (20, 16384), (513, 16384)]


@pytest.fixture(scope="module")
def q():
    import transformer_ffn_block_gb300 as q
    return q


def _backward(q, dy, dr, r, mean, rstd, gain):
    N, C = r.shape
    dx, dg, ds = torch.empty(N, C, dtype=bf16, device="cuda"), torch.empty(C, device="cuda"), torch.empty(C, device="cuda")
    ws = torch.empty(q.qffn_norm_backward_workspace_size(N, C), dtype=torch.uint8, device="cuda")
    q.qffn_layernorm_backward(dx, dg, ds, None, dy.cuda(), None if dr is None else dr.cuda(), r.cuda(), mean.cuda(), rstd.cuda(),
                              gain.cuda(), N, C, False, ws)
    q.qffn_check_status()
    return dx, dg, ds


@pytest.mark.parametrize("N,C", SHAPES)
@pytest.mark.parametrize("offset", [100.0, 200.0])
def test_layernorm_backward_far_from_zero(q, N, C, offset):
    """Means of `offset` standard deviations (the values' bf16 steps are as wide as the deviations then)."""
    g = torch.Generator().manual_seed(N + C)
    sign = torch.where(torch.rand(N, 1, generator=g) < 0.5, -1.0, 1.0)
    r = ((torch.randn(N, C, generator=g) + offset) * sign * (0.5 + torch.rand(N, 1, generator=g))).to(bf16)
    gain = (1.0 + 0.2 * torch.randn(C, generator=g)).to(bf16)
    dy, dr = ((torch.randn(N, C, generator=g) * 0.1).to(bf16) for _ in range(2))
    mean = r.double().mean(1).to(f32)
    rstd = ((r.double() - mean.double()[:, None]).square().mean(1) + 1e-5).rsqrt().to(f32)
    dx, dg, ds = _backward(q, dy, dr, r, mean, rstd, gain)
    d = [t.double() for t in (dy, dr, r, mean, rstd, gain)]
    wdx, wdg, wds, _, _, b_ds = P.norm_backward(*d)
    dy64, _, r64, mu, rs, gain64 = d
    mu, rs = mu[:, None], rs[:, None]
    xh, w = (r64 - mu) * rs, dy64 * gain64
    c1, c2 = (w * xh).mean(1, keepdim=True), w.mean(1, keepdim=True)
    # the difference and the product are rounded once each, 2^-24 of their value; the row sums as in the plain form
    d_xh = 2.0 ** -23 * xh.abs()
    d_c1 = 2.0 ** -19 * (w * xh).abs().mean(1, keepdim=True) + (w.abs() * d_xh).mean(1, keepdim=True)
    d_c2 = 2.0 ** -19 * w.abs().mean(1, keepdim=True)
    b_dx = P.HALF * wdx.abs() + rs * (c1.abs() * d_xh + xh.abs() * d_c1 + d_c2
                                      + 2.0 ** -21 * (w.abs() + c2.abs() + (xh * c1).abs()))
    P.check(dx, wdx, b_dx, "dx")
    # every partial sum is at most the sum of the sizes, each addition half a unit of it
    b_dg = (dy64.abs() * d_xh).sum(0) + (N + 80) * 2.0 ** -24 * (dy64 * xh).abs().sum(0)
    P.check(dg, wdg, b_dg, "dgain")
    P.check(ds, wds, b_ds, "dshift")


@pytest.mark.parametrize("N,C", SHAPES)
@pytest.mark.parametrize("value", [3.0, 1004.0, -0.0117])
def test_layernorm_backward_of_constant_rows(q, N, C, value):
    """r - mean is 0: no gradient of the gain at all."""
    g = torch.Generator().manual_seed(N + C)
    r = torch.full((N, C), value).to(bf16)
    mean, rstd = r[:, 0].float(), torch.full((N,), 1e-5, dtype=torch.float64).rsqrt().to(f32)
    gain, dy = (1.0 + 0.2 * torch.randn(C, generator=g)).to(bf16), (torch.randn(N, C, generator=g) * 0.1).to(bf16)
    dx, dg, ds = _backward(q, dy, None, r, mean, rstd, gain)
    assert (dg == 0).all()
    w = dy.double() * gain.double()
    c2, rs = w.mean(1, keepdim=True), rstd.double()[:, None]
    want = rs * (w - c2)
    P.check(dx, want, P.HALF * want.abs() + rs * (2.0 ** -19 * w.abs().mean(1, keepdim=True) + 2.0 ** -21 * (w.abs() + c2.abs())), "dx")
    P.check(ds, dy.double().sum(0), (N + 80) * 2.0 ** -24 * dy.double().abs().sum(0), "dshift")
