"""GPU parity of the linear and gated layers and of their backward against 64-bit plain forms."""
import pytest
import torch

import plain_ops as P
from test_gpu_canaries import Guarded

pytestmark = pytest.mark.gpu

# one token, fewer rows than a tile, ragged tiles in every direction, lengths of K below and across a
# stage of 128, splits of K, several tiles per CTA pair with a short last wave
SHAPES = [(1, 8, 8), (1, 4096, 1024), (5, 264, 72), (16, 1000, 520), (17, 128, 4104), (33, 520, 136), (129, 256, 2048),
          (200, 776, 1288), (257, 264, 128), (300, 2048, 256), (1100, 5000, 200), (2304, 2568, 136)]
BIG = (4200, 6664, 264)     # 17 x 27 tiles: more than five waves, a short last one
bf16, f32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def q():
    import transformer_ffn_block_gb300 as q
    return q


def _t(seed, *shape, std=1.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std).to(bf16)


def _ws(q, size):
    assert size >= 256
    return Guarded(size)


def _act(q, name):
    return getattr(q, "QFFN_ACT_" + name.upper())


def _linear(q, x, w, bias, res, name, save_z, fp8_scale=None):
    M, N, K = x.shape[0], w.shape[0], x.shape[1]
    out, z = Guarded(M * N * 2), Guarded(M * N * 2)
    size = (q.qffn_linear_fp8_workspace_size if fp8_scale else q.qffn_linear_workspace_size)(M, N, K)
    ws = _ws(q, size)
    b, r = (None if t is None else t.cuda() for t in (bias, res))
    zv = z.view(bf16, M, N) if save_z else None
    if fp8_scale:
        sx, sw = (torch.tensor([v], dtype=f32, device="cuda") for v in fp8_scale)
        q.qffn_linear_fp8(out.view(bf16, M, N), zv, x.cuda(), sx, w.cuda(), sw, b, r, _act(q, name), M, N, K,
                          ws.view(torch.uint8, size))
    else:
        q.qffn_linear(out.view(bf16, M, N), zv, x.cuda(), w.cuda(), b, r, _act(q, name), M, N, K, ws.view(torch.uint8, size))
    q.qffn_check_status()
    for buf, what in ((out, "out"), (z, "z"), (ws, "workspace")):
        buf.check(what)
    return out.view(bf16, M, N), z.view(bf16, M, N)


def _check_linear(q, M, N, K, name, bias, res, save_z, fp8=False):
    x, w = _t(M + K, M, K), _t(N + K, N, K, std=K ** -0.5)
    scale = None
    if fp8:
        x, w, scale = x.to(torch.float8_e4m3fn), (w * 64).to(torch.float8_e4m3fn), (0.5, 1 / 32)
    b, r = (_t(3, N, std=0.5) if bias else None), (_t(4, M, N) if res else None)
    out, z = _linear(q, x, w, b, r, name, save_z, scale)
    d = lambda t: None if t is None else t.double()  # noqa: E731
    want, wz, b_out, b_z = P.linear(d(x), d(w), d(b), d(r), name, scale[0] * scale[1] if fp8 else 1.0)
    P.check(out, want, b_out, "out")
    if save_z:
        P.check(z, wz, b_z, "z")
    # the error of a correctly rounded result is at most HALF per element; sums of independent roundings stay below
    rel = ((out.double().cpu() - want).norm() / want.norm()).item()
    assert rel <= P.HALF, rel


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("name,bias,res,save_z", [("none", False, False, False), ("none", True, True, False),
                                                  ("gelu", True, False, True), ("silu", True, True, True)])
def test_linear(q, M, N, K, name, bias, res, save_z):
    _check_linear(q, M, N, K, name, bias, res, save_z)


@pytest.mark.parametrize("name", list(P.ACTS))
@pytest.mark.parametrize("M", [3, 300])
def test_linear_activations(q, M, name):
    _check_linear(q, M, 520, 264, name, True, True, False)
    _check_linear(q, M, 520, 264, name, False, False, True)


@pytest.mark.parametrize("M,N,K", [(1, 8, 16), (1, 4096, 2048), (7, 264, 80), (33, 520, 4112), (200, 776, 1296),
                                   (300, 2048, 272), (1100, 5000, 208)])
@pytest.mark.parametrize("name,bias,res,save_z", [("none", False, False, False), ("gelu_tanh", True, True, False),
                                                  ("relu", True, False, True), ("silu", False, True, True)])
def test_linear_fp8(q, M, N, K, name, bias, res, save_z):
    _check_linear(q, M, N, K, name, bias, res, save_z, fp8=True)


def test_linear_fp8_equals_the_scaled_gemm(q):
    """Without an epilogue it is the plain FP8 GEMM: the same bits where K is not split."""
    M, N, K = 2304, 2560, 512
    x, w = _t(1, M, K).to(torch.float8_e4m3fn).cuda(), _t(2, N, K).to(torch.float8_e4m3fn).cuda()
    s = torch.tensor([0.25, 0.125], device="cuda")
    a, b = (torch.empty(M, N, dtype=bf16, device="cuda") for _ in range(2))
    ws = torch.empty(q.qffn_linear_fp8_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")
    q.qffn_linear_fp8(a, None, x, s[0:1], w, s[1:2], None, None, q.QFFN_ACT_NONE, M, N, K, ws)
    q.qffn_fp8_gemm_scaled(b, x, s[0:1], w, s[1:2], M, N, K)
    q.qffn_check_status()
    assert torch.equal(a, b)


@pytest.mark.parametrize("name,res,save_z", [("none", True, False), ("gelu", True, True)])
def test_linear_many_waves(q, name, res, save_z):
    _check_linear(q, *BIG, name, True, res, save_z)


@pytest.mark.parametrize("M,K", [(1, 2048), (40, 2048), (300, 264)])
def test_linear_residual_in_place(q, M, K):
    N = 520
    x, w, r = _t(1, M, K).cuda(), _t(2, N, K, std=K ** -0.5).cuda(), _t(3, M, N).cuda()
    ws = torch.empty(q.qffn_linear_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")
    out = torch.empty(M, N, dtype=bf16, device="cuda")
    q.qffn_linear(out, None, x, w, None, r, 0, M, N, K, ws)
    q.qffn_linear(r, None, x, w, None, r, 0, M, N, K, ws)
    q.qffn_check_status()
    assert torch.equal(out, r)


@pytest.mark.parametrize("M", [1, 16, 40, 300])
def test_linear_special_values(q, M):
    """NaN and infinities reach their own rows and columns only; large values saturate as the formulas do."""
    N, K = 264, 136
    x, w = _t(1, M, K), _t(2, N, K, std=0.1)
    bias = torch.zeros(N, dtype=bf16)
    bias[5], bias[6], bias[7], bias[8] = 1e30, -1e30, float("nan"), float("inf")
    for name in ("relu", "gelu", "gelu_tanh", "silu"):
        out, _ = _linear(q, x, w, bias, None, name, False)
        o = out.float().cpu()
        assert torch.allclose(o[:, 5], torch.full((M,), 1e30), rtol=2 ** -7) and (o[:, 6] == 0).all()
        assert o[:, 7].isnan().all() and (o[:, 8] == float("inf")).all()
        assert torch.isfinite(o[:, 9:]).all()
    x[M - 1, 3] = float("nan")
    out, _ = _linear(q, x, w, None, None, "none", False)
    assert out[M - 1].isnan().all() and torch.isfinite(out[:M - 1]).all()


BWD_SHAPES = [(1, 8, 8), (1, 264, 136), (7, 264, 72), (16, 1000, 520), (130, 256, 520), (300, 776, 1288), (1000, 136, 264),
              (1111, 2056, 648), (513, 4096, 2304)]


@pytest.mark.parametrize("M,N,K", BWD_SHAPES)
@pytest.mark.parametrize("name,accumulate,dbias", [("none", False, True), ("none", True, False), ("gelu", True, True),
                                                   ("silu", False, False)])
def test_linear_backward(q, M, N, K, name, accumulate, dbias):
    dout, z, x, w = _t(1, M, N, std=0.1), _t(2, M, N, std=1.5), _t(3, M, K), _t(4, N, K, std=N ** -0.5)
    old, old_b = _t(5, N, K), torch.randn(N, generator=torch.Generator().manual_seed(6))
    dx, dw, db = Guarded(M * K * 2), Guarded(N * K * 2), Guarded(N * 4)
    dw.view(bf16, N, K).copy_(old)
    db.view(f32, N).copy_(old_b)
    size = q.qffn_linear_backward_workspace_size(M, N, K)
    ws = _ws(q, size)
    q.qffn_linear_backward(dx.view(bf16, M, K), dw.view(bf16, N, K), db.view(f32, N) if dbias else None, dout.cuda(),
                           None if name == "none" else z.cuda(), x.cuda(), w.cuda(), _act(q, name), M, N, K, accumulate,
                           ws.view(torch.uint8, size))
    q.qffn_check_status()
    for buf, what in ((dx, "dx"), (dw, "dw"), (db, "dbias"), (ws, "workspace")):
        buf.check(what)
    wdx, wdw, wdb, b_dx, b_dw, b_db = P.linear_backward(dout.double(), z.double(), x.double(), w.double(), name,
                                                        old.double() if accumulate else None)
    P.check(dx.view(bf16, M, K), wdx, b_dx, "dx")
    P.check(dw.view(bf16, N, K), wdw, b_dw, "dw")
    if dbias:
        add = old_b.double() if accumulate else 0
        P.check(db.view(f32, N), wdb + add, b_db + 2.0 ** -23 * (wdb + add).abs(), "dbias")
    else:
        assert torch.equal(db.view(f32, N).cpu(), old_b)


@pytest.mark.parametrize("name", list(P.ACTS))
def test_linear_backward_activations(q, name):
    M, N, K = 70, 136, 72
    dout, z, x, w = _t(1, M, N), _t(2, M, N, std=3.0), _t(3, M, K), _t(4, N, K)
    z[0, :4] = torch.tensor([0.0, -0.0, 30.0, -30.0])
    dx, dw, db = (torch.empty(*s, dtype=t, device="cuda") for s, t in (((M, K), bf16), ((N, K), bf16), ((N,), f32)))
    ws = torch.empty(q.qffn_linear_backward_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")
    q.qffn_linear_backward(dx, dw, db, dout.cuda(), z.cuda(), x.cuda(), w.cuda(), _act(q, name), M, N, K, False, ws)
    q.qffn_check_status()
    wdx, wdw, wdb, b_dx, b_dw, b_db = P.linear_backward(dout.double(), z.double(), x.double(), w.double(), name)
    P.check(dx, wdx, b_dx, "dx")
    P.check(dw, wdw, b_dw, "dw")
    P.check(db, wdb, b_db, "dbias")
    # weight gradient alone: the same bits
    dw2 = torch.empty_like(dw)
    q.qffn_linear_backward(None, dw2, None, dout.cuda(), z.cuda(), x.cuda(), w.cuda(), _act(q, name), M, N, K, False, ws)
    assert torch.equal(dw, dw2)


@pytest.mark.parametrize("name", ["relu", "gelu", "gelu_tanh", "silu"])
def test_linear_backward_far_preactivations(q, name):
    """Where z is huge or infinite the slope is 0 or 1, and a NaN stays in its column."""
    M, N, K = 5, 16, 8
    z = torch.zeros(M, N)
    for c, v in enumerate((1e30, -1e30, 3e38, -3e38, float("inf"), -float("inf"), 90.0, -90.0, 200.0, -200.0, float("nan"))):
        z[:, c] = v
    dout, x, w = _t(1, M, N), _t(2, M, K), _t(3, N, K)
    dx, dw, db = (torch.empty(*s, dtype=t, device="cuda") for s, t in (((M, K), bf16), ((N, K), bf16), ((N,), f32)))
    ws = torch.empty(q.qffn_linear_backward_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")
    q.qffn_linear_backward(dx, dw, db, dout.cuda(), z.to(bf16).cuda(), x.cuda(), w.cuda(), _act(q, name), M, N, K, False, ws)
    q.qffn_check_status()
    db, want = db.cpu().double(), dout.double().sum(0)
    tol = 2.0 ** -20 * dout.double().abs().sum(0)
    for c in range(10):
        assert abs(db[c] - (want[c] if c % 2 == 0 else 0.0)) <= tol[c] + 1e-30, c
    assert db[10].isnan() and dw[10].isnan().all() and torch.isfinite(dw[:10].float()).all()
    at_zero = P.act_grad(torch.zeros(1, dtype=torch.float64), name).item()
    assert bool(((db[11:] - at_zero * want[11:]).abs() <= tol[11:]).all())


@pytest.mark.parametrize("M,C,H", [(1, 8, 8), (1, 1024, 2048), (3, 72, 136), (16, 520, 264), (17, 2048, 72), (40, 136, 1000),
                                   (130, 264, 128), (300, 1024, 776), (700, 264, 3000), (2304, 136, 1280)])
@pytest.mark.parametrize("name", ["silu", "gelu"])
def test_gated_linear(q, M, C, H, name):
    x, w1 = _t(1, M, C), _t(2, 2 * H, C, std=C ** -0.5)
    h = Guarded(M * H * 2)
    size = q.qffn_gated_linear_workspace_size(M, C, H)
    ws = _ws(q, size)
    q.qffn_gated_linear(h.view(bf16, M, H), x.cuda(), w1.cuda(), _act(q, name), M, C, H, ws.view(torch.uint8, size))
    q.qffn_check_status()
    h.check("h")
    ws.check("workspace")
    want, bound, _ = P.gated(x.double(), w1.double(), name)
    P.check(h.view(bf16, M, H), want, bound, "h")
    assert ((h.view(bf16, M, H).double().cpu() - want).norm() / want.norm()).item() <= P.HALF


@pytest.mark.parametrize("M,C,H", [(1, 8, 8), (3, 72, 136), (16, 520, 264), (130, 264, 128), (300, 1024, 776),
                                   (513, 264, 2600), (1111, 648, 1032)])
@pytest.mark.parametrize("name,accumulate", [("silu", False), ("gelu_tanh", True)])
def test_gated_linear_backward(q, M, C, H, name, accumulate):
    dh, x, w1, old = _t(1, M, H, std=0.1), _t(2, M, C), _t(3, 2 * H, C, std=C ** -0.5), _t(4, 2 * H, C)
    dx, dw = Guarded(M * C * 2), Guarded(2 * H * C * 2)
    dw.view(bf16, 2 * H, C).copy_(old)
    size = q.qffn_gated_linear_backward_workspace_size(M, C, H)
    ws = _ws(q, size)
    q.qffn_gated_linear_backward(dx.view(bf16, M, C), dw.view(bf16, 2 * H, C), dh.cuda(), x.cuda(), w1.cuda(),
                                 _act(q, name), M, C, H, accumulate, ws.view(torch.uint8, size))
    q.qffn_check_status()
    for buf, what in ((dx, "dx"), (dw, "dw1"), (ws, "workspace")):
        buf.check(what)
    dz, b_dz, wdx, wdw, b_dx, b_dw = P.gated_backward(dh.double(), x.double(), w1.double(), name,
                                                      old.double() if accumulate else None)
    P.check(ws.view(torch.uint8, size)[:M * 2 * H * 2].view(bf16).view(M, 2 * H), dz, b_dz, "d_gu")
    P.check(dx.view(bf16, M, C), wdx, b_dx, "dx")
    P.check(dw.view(bf16, 2 * H, C), wdw, b_dw, "dw1")


@pytest.mark.parametrize("name", list(P.ACTS))
@pytest.mark.parametrize("M", [3, 300])
def test_gated_activations(q, M, name):
    C, H = 136, 264
    dh, x, w1 = _t(1, M, H), _t(2, M, C), _t(3, 2 * H, C, std=C ** -0.5)
    h, dx, dw = (torch.empty(*s, dtype=bf16, device="cuda") for s in ((M, H), (M, C), (2 * H, C)))
    ws = torch.empty(q.qffn_gated_linear_backward_workspace_size(M, C, H), dtype=torch.uint8, device="cuda")
    q.qffn_gated_linear(h, x.cuda(), w1.cuda(), _act(q, name), M, C, H,
                        torch.empty(q.qffn_gated_linear_workspace_size(M, C, H), dtype=torch.uint8, device="cuda"))
    q.qffn_gated_linear_backward(dx, dw, dh.cuda(), x.cuda(), w1.cuda(), _act(q, name), M, C, H, False, ws)
    q.qffn_check_status()
    want, bound, _ = P.gated(x.double(), w1.double(), name)
    P.check(h, want, bound, "h")
    _, _, wdx, wdw, b_dx, b_dw = P.gated_backward(dh.double(), x.double(), w1.double(), name)
    P.check(dx, wdx, b_dx, "dx")
    P.check(dw, wdw, b_dw, "dw1")


def test_no_rows(q):
    N, K = 272, 136
    w = _t(1, N, K).cuda()
    p = w.data_ptr()
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    big = torch.empty(max(q.qffn_linear_backward_workspace_size(0, N, K),
                          q.qffn_gated_linear_backward_workspace_size(0, K, N // 2)), dtype=torch.uint8, device="cuda")
    q.qffn_linear(p, None, p, w, None, None, 0, 0, N, K, ws)
    q.qffn_gated_linear(p, p, w, 4, 0, K, N // 2, ws)
    dw, db = _t(2, N, K).cuda(), torch.ones(N, device="cuda")
    keep = dw.clone()
    q.qffn_linear_backward(None, dw, db, p, p, p, w, 2, 0, N, K, True, big)
    q.qffn_gated_linear_backward(None, dw, p, p, w, 4, 0, K, N // 2, True, big)
    assert torch.equal(dw, keep) and (db == 1).all()
    q.qffn_linear_backward(None, dw, db, p, p, p, w, 2, 0, N, K, False, big)
    assert (dw == 0).all() and (db == 0).all()
    dw.copy_(keep)
    q.qffn_gated_linear_backward(None, dw, p, p, w, 4, 0, K, N // 2, False, big)
    assert (dw == 0).all()
