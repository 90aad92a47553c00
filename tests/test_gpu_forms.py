"""The norm, linear and gated operators at sizes that reach each form of their kernels (the number of rows and
the lengths choose it), past 2^31 elements, in place and with special values."""
import pytest
import torch

import plain_ops as P
from test_gpu_linear import (_act, _check_linear, _linear, _t, bf16, f32, q,  # noqa: F401
                             test_gated_linear, test_gated_linear_backward, test_linear_backward)
from test_gpu_norm import _empty, _rows, _vec, test_layernorm, test_norm_backward

(_gated, _gated_backward, _linear_backward, _layernorm, _norm_backward) = (
    test_gated_linear, test_gated_linear_backward, test_linear_backward, test_layernorm, test_norm_backward)
del test_gated_linear, test_gated_linear_backward, test_linear_backward, test_layernorm, test_norm_backward

pytestmark = pytest.mark.gpu

# weights streamed by 8, 16 or 32 warps per block; few rows of one to four tiles over 1, 2, 4 and 8 parts of K,
# one or two blocks per SM; units of 256, 128 and 64 columns, over parts of K, with halves in the last wave
FORWARD = [(1, 8, 2072), (1, 8, 4104), (9, 8, 2208), (37, 8664, 8), (133, 9936, 8), (271, 6416, 8), (17, 9168, 544),
           (131, 2792, 3280), (285, 2488, 1824), (33, 2232, 1712), (130, 888, 1712), (296, 344, 2200), (33, 1072, 4392),
           (200, 480, 2312), (487, 168, 2960), (776, 2312, 8), (517, 6880, 8), (20, 4624, 8336), (66, 5264, 264),
           (533, 408, 4568), (1316, 24, 7032)]
FORWARD_FP8 = [(1, 8, 4112), (1, 8, 8272), (9, 8, 4128), (35, 5672, 16), (135, 9952, 16), (17, 2320, 2320), (141, 2536, 7152),
               (305, 112, 5216), (419, 56, 6672), (33, 5072, 1008), (324, 1696, 8848), (808, 288, 8720), (782, 24, 7536)]
GATED = [(1, 2056, 8), (1, 4112, 8), (10, 2104, 8), (33, 8, 4552), (134, 8, 5272), (17, 784, 3744), (138, 3272, 1456),
         (130, 1928, 392), (266, 2528, 176), (549, 8, 3424), (24, 7600, 2312), (34, 504, 2488), (787, 4304, 144),
         (937, 3488, 40)]
# input gradient few rows over parts of K, whole, narrow and split units; weight gradient whole, narrow and split,
# and begun on the SMs that the input gradient leaves free
BACKWARD = [(135, 1432, 3112), (273, 1592, 1808), (419, 2296, 1264), (130, 968, 8), (392, 2024, 8), (137, 8, 9776),
            (524, 8, 6664), (2, 4008, 4624), (517, 2328, 8), (8, 264, 10696), (3240, 8, 3384), (2336, 8, 8),
            (700, 5000, 2056), (1111, 4104, 2056)]
GATED_BACKWARD = [(135, 8, 5192), (139, 3312, 1248), (414, 1992, 8), (534, 8, 3384), (2, 4008, 2344), (533, 3744, 264),
                  (524, 2800, 8), (35, 520, 2520), (700, 2056, 2504)]


# the same with the operands exchanged (columns and rows of several tiles), and every split of few rows in each number
# of tiles
FORWARD += [(776, 2312, 8), (653, 3104, 8), (66, 6640, 136), (33, 9928, 8), (19, 5008, 4696), (270, 3144, 8176),
            (165, 584, 2192), (257, 488, 2104), (410, 432, 2576), (372, 312, 1992), (1486, 2848, 8), (1472, 10032, 8),
            (1145, 7352, 80), (803, 1256, 136), (338, 2504, 8), (104, 792, 2632)]
FORWARD_FP8 += [(771, 2392, 16), (772, 2648, 16), (68, 6472, 144), (18, 11336, 16), (154, 264, 4400), (279, 176, 4208),
                (421, 416, 4896), (18, 1440, 4064), (133, 232, 4880), (322, 104, 4768), (1488, 2424, 16),
                (1467, 7656, 16), (1160, 7344, 144), (816, 1248, 272), (516, 1632, 16), (9, 8, 16)]
GATED += [(17, 8, 10232), (267, 8, 2448), (17, 2520, 2440), (281, 5160, 1464), (33, 1760, 1072), (258, 2072, 232),
          (421, 2480, 264), (34, 4680, 464), (234, 1992, 248), (499, 2416, 104), (260, 8, 8056), (70, 8, 2928),
          (99, 2600, 392)]
BACKWARD += [(3384, 8, 3400), (1, 4912, 4904), (131, 1952, 8), (272, 1960, 8), (503, 2064, 16), (259, 2360, 8),
             (1463, 8, 2456), (1454, 72, 5968), (1, 5256, 5080), (588, 8, 3080), (796, 8, 2592), (68, 136, 6728)]
GATED_BACKWARD += [(1, 8, 9840), (257, 8, 2480), (1, 1992, 2448), (279, 4728, 1480), (1, 976, 8), (147, 1928, 8),
                   (275, 2144, 8), (393, 2464, 216), (1, 2000, 8), (131, 2280, 8), (259, 2008, 8), (267, 8, 7376),
                   (1, 5136, 2800), (65, 8, 2616), (71, 3088, 8)]


@pytest.mark.parametrize("M,N,K", FORWARD)
@pytest.mark.parametrize("name,bias,res,save_z", [("none", False, False, False), ("gelu", True, True, True)])
def test_linear_forms(q, M, N, K, name, bias, res, save_z):  # noqa: F811
    _check_linear(q, M, N, K, name, bias, res, save_z)


@pytest.mark.parametrize("M,N,K", FORWARD_FP8)
@pytest.mark.parametrize("name,bias,res,save_z", [("none", False, False, False), ("silu", True, True, True)])
def test_linear_fp8_forms(q, M, N, K, name, bias, res, save_z):  # noqa: F811
    _check_linear(q, M, N, K, name, bias, res, save_z, fp8=True)


@pytest.mark.parametrize("M,N,K", [(16, 520, 264), (133, 2008, 8), (33, 1072, 4392), (101, 4312, 8), (533, 408, 4568),
                                   (700, 3104, 264), (1100, 5000, 200)])
def test_linear_residual_in_place_in_each_form(q, M, N, K):  # noqa: F811
    x, w, r, b = _t(1, M, K).cuda(), _t(2, N, K, std=K ** -0.5).cuda(), _t(3, M, N).cuda(), _t(4, N).cuda()
    ws = torch.empty(q.qffn_linear_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")
    out, z, z2 = _empty(M, N), _empty(M, N), _empty(M, N)
    q.qffn_linear(out, z, x, w, b, r, q.QFFN_ACT_GELU, M, N, K, ws)
    q.qffn_linear(r, z2, x, w, b, r, q.QFFN_ACT_GELU, M, N, K, ws)
    q.qffn_check_status()
    assert torch.equal(out, r) and torch.equal(z, z2)


@pytest.mark.parametrize("M,N,K", [(1100, 5008, 208), (803, 1256, 144), (101, 4312, 16), (1472, 10032, 16), (300, 2048, 272),
                                   (257, 264, 8848)])
@pytest.mark.parametrize("fp8", [False, True])
def test_linear_residual_alone(q, M, N, K, fp8):  # noqa: F811
    _check_linear(q, M, N, K, "none", False, True, False, fp8=fp8)


@pytest.mark.parametrize("M,C,H", GATED)
def test_gated_linear_forms(q, M, C, H):  # noqa: F811
    _gated(q, M, C, H, "silu")


@pytest.mark.parametrize("M,N,K", BACKWARD)
@pytest.mark.parametrize("name,accumulate,dbias", [("none", True, False), ("silu", False, True)])
def test_linear_backward_forms(q, M, N, K, name, accumulate, dbias):  # noqa: F811
    _linear_backward(q, M, N, K, name, accumulate, dbias)


@pytest.mark.parametrize("M,C,H", GATED_BACKWARD)
@pytest.mark.parametrize("accumulate", [False, True])
def test_gated_linear_backward_forms(q, M, C, H, accumulate):  # noqa: F811
    _gated_backward(q, M, C, H, "silu", accumulate)


@pytest.mark.parametrize("N,C", [(1217, 1000), (1300, 2048), (1300, 4096), (1250, 8200), (1217, 16384), (1217, 264), (1219, 8)])
@pytest.mark.parametrize("residual", [False, True])
def test_layernorm_many_rows(q, N, C, residual):  # noqa: F811
    _layernorm(q, N, C, residual, True)


@pytest.mark.parametrize("N,C", [(257, 8), (700, 264), (2500, 264), (5000, 512), (513, 1000), (700, 1032), (1300, 2048),
                                 (600, 8192), (515, 8200), (513, 16384)])
@pytest.mark.parametrize("rms,dres,accumulate", [(False, True, False), (True, False, True), (True, True, False)])
def test_norm_backward_many_rows(q, N, C, rms, dres, accumulate):  # noqa: F811
    _norm_backward(q, N, C, rms, dres, accumulate)


@pytest.mark.parametrize("N,C", [(1, 264), (3, 16384), (37, 2048), (300, 4096), (300, 512), (700, 1000)])
@pytest.mark.parametrize("rms", [False, True])
def test_norm_backward_in_place(q, N, C, rms):  # noqa: F811
    """dx in the place of dy or dres.  With dy few rows too take the form of many, whose row sums are added in
    another order: within the bounds of both, not the same bits."""
    g = torch.Generator().manual_seed(5)
    r, gain = _rows(N, C, 9), _vec(C, 4, mean=1.0)
    dy, dr = ((torch.randn(N, C, generator=g) * 0.1).to(bf16) for _ in range(2))
    mean = None if rms else r.float().mean(1)
    rstd = ((r.float() - (0 if rms else mean[:, None])).square().mean(1) + 1e-5).rsqrt()
    ws = torch.empty(q.qffn_norm_backward_workspace_size(N, C), dtype=torch.uint8, device="cuda")
    d = lambda t: None if t is None else t.double()  # noqa: E731
    wdx, wdg, wds, b_dx, b_dg, b_ds = P.norm_backward(d(dy), d(dr), d(r), d(mean), d(rstd), d(gain))
    for inplace in ("dy", "dres"):
        t = {"dy": dy.cuda(), "dres": dr.cuda()}
        dx, dg, ds = t[inplace], _empty(C, dtype=f32), _empty(C, dtype=f32)
        if rms:
            q.qffn_rmsnorm_backward(dx, dg, None, t["dy"], t["dres"], r.cuda(), rstd.cuda(), gain.cuda(), N, C, False, ws)
        else:
            q.qffn_layernorm_backward(dx, dg, ds, None, t["dy"], t["dres"], r.cuda(), mean.cuda(), rstd.cuda(), gain.cuda(),
                                      N, C, False, ws)
            P.check(ds, wds, b_ds, "dshift")
        q.qffn_check_status()
        P.check(dx, wdx, b_dx, "dx")
        P.check(dg, wdg, b_dg, "dgain")


@pytest.mark.parametrize("M", [1, 16, 40, 300, 600])
def test_gated_special_values(q, M):  # noqa: F811
    """A NaN in a row of x, infinities in a row of w1: their own row and columns only, in every product."""
    C, H = 136, 264
    x, w1, dh = _t(1, M, C), _t(2, 2 * H, C, std=0.1), _t(3, M, H)
    x[M - 1, 3] = float("nan")
    w1[7] = float("nan")                   # gate of column 7
    w1[H + 9] = float("nan")               # up of column 9
    h, dx, dw = _empty(M, H), _empty(M, C), _empty(2 * H, C)
    size = q.qffn_gated_linear_backward_workspace_size(M, C, H)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    q.qffn_gated_linear(h, x.cuda(), w1.cuda(), q.QFFN_ACT_SILU, M, C, H,
                        torch.empty(q.qffn_gated_linear_workspace_size(M, C, H), dtype=torch.uint8, device="cuda"))
    nan = h.isnan().cpu()
    want = torch.zeros(M, H, dtype=torch.bool)
    want[M - 1], want[:, 7], want[:, 9] = True, True, True
    assert torch.equal(nan, want)
    w1[7], w1[H + 9] = 0.5, 0.5            # the gradient: the NaN row of x only
    q.qffn_gated_linear_backward(dx, dw, dh.cuda(), x.cuda(), w1.cuda(), q.QFFN_ACT_SILU, M, C, H, False, ws)
    q.qffn_check_status()
    assert dx[M - 1].isnan().all() and torch.isfinite(dx[:M - 1].float()).all()
    assert dw.isnan().all()                # each weight's gradient sums over every row


@pytest.mark.parametrize("M", [1, 40, 300, 600])
def test_linear_backward_special_values(q, M):  # noqa: F811
    """A NaN in dout: its row of dx and its column's row of dw and element of dbias."""
    N, K = 264, 136
    dout, x, w = _t(1, M, N), _t(2, M, K), _t(3, N, K)
    dout[M - 1, 5] = float("nan")
    dx, dw, db = _empty(M, K), _empty(N, K), _empty(N, dtype=f32)
    ws = torch.empty(q.qffn_linear_backward_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")
    q.qffn_linear_backward(dx, dw, db, dout.cuda(), None, x.cuda(), w.cuda(), q.QFFN_ACT_NONE, M, N, K, False, ws)
    q.qffn_check_status()
    for t, i in ((dx, M - 1), (dw, 5), (db, 5)):
        assert t[i].isnan().all()
        t[i] = 0
        assert torch.isfinite(t.float()).all()


# ---- offsets past 2^31 elements: rows at the start, around that element and at the end
def _some_rows(M, per_row):
    edge = 2 ** 31 // per_row
    return sorted({0, 1, edge - 1, edge, edge + 1, M // 2, M - 257, M - 1} | set(range(edge // 2, edge // 2 + 20)))


def _on_device(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(*shape, dtype=bf16, device="cuda").normal_(0.0, std, generator=g)


def test_linear_past_2_31_elements(q):  # noqa: F811
    M, N, K = 530001, 4104, 64
    x, res = _on_device(1, M, K), _on_device(2, M, N)
    w, b = _t(3, N, K, std=K ** -0.5), _t(4, N)
    ws = torch.empty(q.qffn_linear_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")
    rows = torch.tensor(_some_rows(M, N))
    before = res[rows.cuda()].cpu().double()
    z = torch.empty(M, N, dtype=bf16, device="cuda")
    q.qffn_linear(res, z, x, w.cuda(), b.cuda(), res, q.QFFN_ACT_RELU, M, N, K, ws)
    q.qffn_check_status()
    want, wz, b_out, b_z = P.linear(x[rows.cuda()].cpu().double(), w.double(), b.double(), before, "relu")
    P.check(res[rows.cuda()], want, b_out, "out")
    P.check(z[rows.cuda()], wz, b_z, "z")


def test_linear_backward_past_2_31_elements(q):  # noqa: F811
    M, N, K = 530001, 4104, 64
    dout, z, x = _on_device(1, M, N, std=0.1), _on_device(2, M, N), _on_device(3, M, K)
    w = _t(4, N, K, std=N ** -0.5)
    ws = torch.empty(q.qffn_linear_backward_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")
    dx, dw, db = _empty(M, K), _empty(N, K), _empty(N, dtype=f32)
    q.qffn_linear_backward(dx, dw, db, dout, z, x, w.cuda(), q.QFFN_ACT_RELU, M, N, K, False, ws)
    q.qffn_check_status()
    rows = torch.tensor(_some_rows(M, N)).cuda()
    wdx, _, _, b_dx, _, _ = P.linear_backward(*(t.cpu().double() for t in (dout[rows], z[rows], x[rows], w)), "relu")
    P.check(dx[rows], wdx, b_dx, "dx")
    # the sums over all rows, for eight outputs (relu: dz is dout or 0, no rounding of its own)
    cols = torch.tensor([0, 1, 255, 256, 2051, 4095, 4096, 4103]).cuda()
    dz = dout[:, cols].double() * (z[:, cols] > 0)
    wdw, a_dw = dz.t() @ x.double(), dz.abs().t() @ x.double().abs()
    P.check(dw[cols], wdw.cpu(), (P.HALF * wdw.abs() + 2 * M * P.ACC * a_dw).cpu(), "dw")
    P.check(db[cols], dz.sum(0).cpu(), ((M + 80) * 2.0 ** -24 * dz.abs().sum(0)).cpu(), "dbias")


def test_gated_past_2_31_elements(q):  # noqa: F811
    M, C, H = 530001, 64, 4104
    x, dh = _on_device(1, M, C), _on_device(2, M, H, std=0.1)
    w1 = _t(3, 2 * H, C, std=C ** -0.5)
    ws = torch.empty(q.qffn_gated_linear_backward_workspace_size(M, C, H), dtype=torch.uint8, device="cuda")
    h, dx, dw = torch.empty(M, H, dtype=bf16, device="cuda"), _empty(M, C), _empty(2 * H, C)
    q.qffn_gated_linear(h, x, w1.cuda(), q.QFFN_ACT_SILU, M, C, H,
                        torch.empty(q.qffn_gated_linear_workspace_size(M, C, H), dtype=torch.uint8, device="cuda"))
    q.qffn_gated_linear_backward(dx, dw, dh, x, w1.cuda(), q.QFFN_ACT_SILU, M, C, H, False, ws)
    q.qffn_check_status()
    rows = torch.tensor(_some_rows(M, H)).cuda()
    xr, dr = x[rows].cpu().double(), dh[rows].cpu().double()
    want, bound, _ = P.gated(xr, w1.double(), "silu")
    P.check(h[rows], want, bound, "h")
    dz, b_dz, wdx, _, b_dx, _ = P.gated_backward(dr, xr, w1.double(), "silu")
    P.check(dx[rows], wdx, b_dx, "dx")
    P.check(ws[:M * 2 * H * 2].view(bf16).view(M, 2 * H)[rows], dz, b_dz, "d_gu")


def test_norms_past_2_31_elements(q):  # noqa: F811
    N, C = 530001, 4104
    x, res = _on_device(1, N, C), _on_device(2, N, C)
    gain, shift = _vec(C, 3, mean=1.0), _vec(C, 4)
    y, mean, rstd = torch.empty(N, C, dtype=bf16, device="cuda"), _empty(N, dtype=f32), _empty(N, dtype=f32)
    q.qffn_layernorm_absmax(res, y, mean, rstd, None, res, x, gain.cuda(), shift.cuda(), 1e-5, N, C)
    rows = torch.tensor(_some_rows(N, C)).cuda()
    r = res[rows].cpu()
    from test_gpu_norm import _check_forward
    _check_forward(y[rows], mean[rows], rstd[rows], r, gain, shift, 1e-5)
    dg, ds = _empty(C, dtype=f32), _empty(C, dtype=f32)
    ws = torch.empty(q.qffn_norm_backward_workspace_size(N, C), dtype=torch.uint8, device="cuda")
    dy, dr = y[rows].cpu(), x[rows].cpu()
    cols = torch.tensor([0, 1, 255, 256, 2051, 4095, 4096, 4103]).cuda()
    d8 = y[:, cols].double()               # y becomes dx below
    q.qffn_layernorm_backward(y, dg, ds, None, y, x, res, mean, rstd, gain.cuda(), N, C, False, ws)
    q.qffn_check_status()
    wdx, _, _, b_dx, _, _ = P.norm_backward(dy.double(), dr.double(), r.double(), mean[rows].cpu().double(),
                                            rstd[rows].cpu().double(), gain.double())
    P.check(y[rows], wdx, b_dx, "dx")
    mu, rs = mean.double()[:, None], rstd.double()[:, None]
    r8 = res[:, cols].double()
    xh = (r8 - mu) * rs
    # as in the plain form: the rounding of xhat, and the fp32 sums over the rows
    b_dg = (d8.abs() * 2.0 ** -22 * (r8.abs() + mu.abs()) * rs).sum(0) + (N + 80) * 2.0 ** -24 * (d8 * xh).abs().sum(0)
    P.check(dg[cols], (d8 * xh).sum(0).cpu(), b_dg.cpu(), "dgain")
    P.check(ds[cols], d8.sum(0).cpu(), ((N + 80) * 2.0 ** -24 * d8.abs().sum(0)).cpu(), "dshift")
