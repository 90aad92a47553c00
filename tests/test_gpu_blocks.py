"""The norm, linear and gated operators run together as a transformer's feed-forward half uses them,
forward and backward, and under streams and CUDA graphs."""
import numpy as np
import pytest
import torch

import oracle
import plain_ops as P
from ffn_inputs import random_bf16
from gpu_util import dev

pytestmark = pytest.mark.gpu
bf16, f32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def q():
    import transformer_ffn_block_gb300 as q
    return q


def _t(seed, *shape, std=1.0, mean=0.0):
    return (torch.randn(*shape, generator=torch.Generator().manual_seed(seed)) * std + mean).to(bf16)


def _new(*shape, dtype=bf16):
    return torch.full(shape, float("nan"), dtype=dtype, device="cuda")


def _ws(size):
    return torch.empty(size, dtype=torch.uint8, device="cuda")


def _rel(got, want):
    return ((got.double().cpu() - want).norm() / want.norm()).item()


# Independent bf16 roundings of relative size at most HALF along the way add in the mean square; no
# step of these chains amplifies a random error by more than about two: 16 HALF bounds them all.
CHAIN = 16 * P.HALF


class Mlp:
    """Pre-norm block: out = r + act(ln(r) W1^T + b1) W2^T + b2 with r = res + x."""

    def __init__(self, q, M, C, H, act="gelu", seed=0):
        self.q, self.M, self.C, self.H, self.act = q, M, C, H, act
        self.host = dict(x=_t(seed + 1, M, C), res=_t(seed + 2, M, C), gain=_t(seed + 3, C, std=0.1, mean=1.0),
                         shift=_t(seed + 4, C, std=0.1), w1=_t(seed + 5, H, C, std=C ** -0.5), b1=_t(seed + 6, H, std=0.1),
                         w2=_t(seed + 7, C, H, std=H ** -0.5), b2=_t(seed + 8, C, std=0.1), dout=_t(seed + 9, M, C, std=0.1))
        self.d = {k: v.cuda() for k, v in self.host.items()}
        self.o = dict(r=_new(M, C), y=_new(M, C), mean=_new(M, dtype=f32), rstd=_new(M, dtype=f32), z=_new(M, H), h=_new(M, H),
                      out=_new(M, C), dh=_new(M, H), dw2=_new(C, H), db2=_new(C, dtype=f32), dy=_new(M, C), dw1=_new(H, C),
                      db1=_new(H, dtype=f32), dx=_new(M, C), dgain=_new(C, dtype=f32), dshift=_new(C, dtype=f32))
        size = max(q.qffn_linear_workspace_size(M, H, C), q.qffn_linear_workspace_size(M, C, H),
                   q.qffn_linear_backward_workspace_size(M, H, C), q.qffn_linear_backward_workspace_size(M, C, H),
                   q.qffn_norm_backward_workspace_size(M, C))
        self.ws = _ws(size)

    def step(self, stream=None):
        q, d, o, M, C, H, ws = self.q, self.d, self.o, self.M, self.C, self.H, self.ws
        act = getattr(q, "QFFN_ACT_" + self.act.upper())
        q.qffn_layernorm_absmax(o["r"], o["y"], o["mean"], o["rstd"], None, d["res"], d["x"], d["gain"], d["shift"], 1e-5, M, C,
                                stream=stream)
        q.qffn_linear(o["h"], o["z"], o["y"], d["w1"], d["b1"], None, act, M, H, C, ws, stream=stream)
        q.qffn_linear(o["out"], None, o["h"], d["w2"], d["b2"], o["r"], q.QFFN_ACT_NONE, M, C, H, ws, stream=stream)
        q.qffn_linear_backward(o["dh"], o["dw2"], o["db2"], d["dout"], None, o["h"], d["w2"], q.QFFN_ACT_NONE, M, C, H, False, ws,
                               stream=stream)
        q.qffn_linear_backward(o["dy"], o["dw1"], o["db1"], o["dh"], o["z"], o["y"], d["w1"], act, M, H, C, False, ws, stream=stream)
        q.qffn_layernorm_backward(o["dx"], o["dgain"], o["dshift"], None, o["dy"], d["dout"], o["r"], o["mean"], o["rstd"],
                                  d["gain"], M, C, False, ws, stream=stream)

    def want(self):
        h = {k: v.double() for k, v in self.host.items()}
        leaves = {k: h[k].clone().requires_grad_() for k in ("x", "gain", "shift", "w1", "b1", "w2", "b2")}
        r = leaves["x"] + h["res"]
        y, _, _ = P.layernorm(r, leaves["gain"], leaves["shift"], 1e-5)
        out = r + P.act(y @ leaves["w1"].t() + leaves["b1"], self.act) @ leaves["w2"].t() + leaves["b2"]
        out.backward(h["dout"])
        g = {("dx" if k == "x" else "d" + k): v.grad for k, v in leaves.items()}
        return dict(out=out.detach(), **g)


@pytest.mark.parametrize("M,C,H", [(1, 264, 1032), (20, 264, 1032), (77, 512, 2048), (300, 264, 1032), (1111, 1024, 4096)])
@pytest.mark.parametrize("act", ["gelu", "silu"])
def test_layernorm_mlp_step(q, M, C, H, act):
    """Forward and backward of the whole block against autograd in 64 bits."""
    b = Mlp(q, M, C, H, act)
    b.step()
    q.qffn_check_status()
    for k, v in b.want().items():
        assert _rel(b.o[k], v) <= CHAIN, k


@pytest.mark.parametrize("M,C,H", [(1, 264, 520), (50, 512, 1536), (700, 1024, 2816)])
def test_rmsnorm_gated_step(q, M, C, H):
    """r = res + x; out = r + (act(g) * u) W2^T with g, u = rms(r) W1^T: forward and backward."""
    host = dict(x=_t(1, M, C), res=_t(2, M, C), gain=_t(3, C, std=0.1, mean=1.0), w1=_t(4, 2 * H, C, std=C ** -0.5),
                w2=_t(5, C, H, std=H ** -0.5), dout=_t(6, M, C, std=0.1))
    d = {k: v.cuda() for k, v in host.items()}
    r, y, h, out, dh, dw2, dy, dw1, dx = (_new(*s) for s in ((M, C), (M, C), (M, H), (M, C), (M, H), (C, H), (M, C), (2 * H, C), (M, C)))
    rstd, dgain, stats = _new(M, dtype=f32), _new(C, dtype=f32), torch.zeros(2, device="cuda")
    q.qffn_rmsnorm_absmax(r, y, rstd, None, d["res"], d["x"], d["gain"], 1e-5, M, C)
    q.qffn_gated_linear(h, y, d["w1"], q.QFFN_ACT_SILU, M, C, H, _ws(q.qffn_gated_linear_workspace_size(M, C, H)))
    q.qffn_linear(out, None, h, d["w2"], None, r, q.QFFN_ACT_NONE, M, C, H, _ws(q.qffn_linear_workspace_size(M, C, H)))
    q.qffn_linear_backward(dh, dw2, None, d["dout"], None, h, d["w2"], q.QFFN_ACT_NONE, M, C, H, False,
                           _ws(q.qffn_linear_backward_workspace_size(M, C, H)))
    q.qffn_gated_linear_backward(dy, dw1, dh, y, d["w1"], q.QFFN_ACT_SILU, M, C, H, False,
                                 _ws(q.qffn_gated_linear_backward_workspace_size(M, C, H)))
    q.qffn_rmsnorm_backward(dx, dgain, stats, dy, d["dout"], r, rstd, d["gain"], M, C, False,
                            _ws(q.qffn_norm_backward_workspace_size(M, C)))
    q.qffn_check_status()
    v = {k: t.double() for k, t in host.items()}
    lv = {k: v[k].clone().requires_grad_() for k in ("x", "gain", "w1", "w2")}
    rr = lv["x"] + v["res"]
    yy = rr / torch.sqrt((rr * rr).mean(1, keepdim=True) + 1e-5) * lv["gain"]
    oo = rr + P.gated(yy, lv["w1"], "silu")[0] @ lv["w2"].t()
    oo.backward(v["dout"])
    for name, got, want in (("out", out, oo.detach()), ("dx", dx, lv["x"].grad), ("dgain", dgain, lv["gain"].grad),
                            ("dw1", dw1, lv["w1"].grad), ("dw2", dw2, lv["w2"].grad)):
        assert _rel(got, want) <= CHAIN, name
    assert stats[0].item() == dx.float().abs().max().item()


def test_fp8_block_through_the_norm(q):
    """The FP8 feed-forward block with its residual fused into the down projection, and its backward
    finished by the norm's, whose abs-max the layer before quantises the gradient with."""
    N, C, H = 256, 256, 768
    x, res, gain = random_bf16((N, C), seed=1), random_bf16((N, C), seed=2), random_bf16((C,), seed=3)
    w1q, w1s = oracle.quantize_tensor(random_bf16((2 * H, C), seed=4, std=0.05))
    w2q, w2s = oracle.quantize_tensor(random_bf16((C, H), seed=5, std=0.05))
    r, y, h = (torch.empty(N, w, dtype=bf16, device="cuda") for w in (C, C, H))
    yq, hq = (torch.empty(N, w, dtype=torch.uint8, device="cuda") for w in (C, H))
    rstd = _new(N, dtype=f32)
    sty, sth, stg, std_ = (torch.zeros(2, device="cuda") for _ in range(4))
    sc = torch.tensor([w1s, w2s], dtype=f32, device="cuda")
    w1, w2, gaind = dev(w1q), dev(w2q), dev(gain)
    q.qffn_rmsnorm_absmax(r, y, rstd, sty, dev(res), dev(x), gaind, 1e-5, N, C)
    q.qffn_quantize(yq, sty, y, N * C)
    q.qffn_gate_up_swiglu(h, sth, yq, sty[1:], w1, sc[0:1], N, C, H)
    q.qffn_quantize(hq, sth, h, N * H)
    out, plain = _new(N, C), _new(N, C)
    q.qffn_linear_fp8(out, None, hq, sth[1:], w2, sc[1:], None, r, q.QFFN_ACT_NONE, N, C, H,
                      _ws(q.qffn_linear_fp8_workspace_size(N, C, H)))
    q.qffn_fp8_gemm_scaled(plain, hq, sth[1:], w2, sc[1:], N, C, H)
    # the fused sum is rounded once, the two calls' twice
    two = plain.double() + r.double()
    assert bool(((out.double() - two).abs() <= P.HALF * (out.double().abs() + plain.double().abs()) + 1e-30).all())
    dout = dev(random_bf16((N, C), seed=6, std=1e-2)).view(bf16)
    d_ln2, dw1, dw2 = _new(N, C), _new(2 * H, C), _new(C, H)
    q.qffn_absmax(stg, dout, N * C)
    q.qffn_ffn_backward(d_ln2, dw1, dw2, stg, std_, dout, yq, sty[1:], hq, sth[1:], w1, sc[0:1], w2, sc[1:], N, C, H, False,
                        _ws(q.qffn_ffn_backward_workspace_size(N, C, H)))
    dx, dgain, stx = _new(N, C), _new(C, dtype=f32), torch.full((2,), 3.0, device="cuda")
    q.qffn_rmsnorm_backward(dx, dgain, stx, d_ln2, dout, r, rstd, gaind, N, C, False,
                            _ws(q.qffn_norm_backward_workspace_size(N, C)))
    q.qffn_check_status()
    g64 = torch.from_numpy(np.ascontiguousarray(oracle.bf16_to_f64(gain)))
    wdx, wdg, _, b_dx, b_dg, _ = P.norm_backward(d_ln2.double().cpu(), dout.double().cpu(), r.double().cpu(), None,
                                                 rstd.double().cpu(), g64)
    P.check(dx, wdx, b_dx, "dx")
    P.check(dgain, wdg, b_dg, "dgain")
    assert stx[0].item() == dx.float().abs().max().item() and stx[1].item() == 3.0


SIZES = [(1, 264, 1032), (40, 512, 2048), (333, 512, 2048), (1111, 264, 1032)]


@pytest.mark.parametrize("M,C,H", SIZES)
def test_steps_on_two_streams_at_once(q, M, C, H):
    """Two blocks with their own buffers, enqueued alternately on two streams, give the bits each gives alone."""
    blocks = [Mlp(q, M, C, H, seed=10), Mlp(q, M, C, H, seed=30)]
    alone = []
    for b in blocks:
        b.step()
        torch.cuda.synchronize()
        alone.append({k: v.clone() for k, v in b.o.items()})
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for b, s in zip(blocks, streams):
            b.step(stream=s)
    torch.cuda.synchronize()
    q.qffn_check_status()
    for b, want in zip(blocks, alone):
        for k, v in want.items():
            assert torch.equal(b.o[k], v), k


@pytest.mark.parametrize("M,C,H", SIZES)
def test_captured_steps_share_a_workspace(q, M, C, H):
    """Two captured steps with one workspace, replayed one after the other on one stream and on new
    inputs, equal the eager calls bit for bit; an eager step between the replays is left alone too."""
    a, b = Mlp(q, M, C, H, seed=50), Mlp(q, M, C, H, act="silu", seed=70)
    b.ws = a.ws
    fresh = Mlp(q, M, C, H, seed=90)
    a.step()
    b.step()
    torch.cuda.synchronize()
    graphs = []
    for m in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            m.step()
        graphs.append(g)
    for m in (a, b):                                   # other inputs in the same buffers
        for k in ("x", "res", "dout"):
            m.d[k].copy_(fresh.d[k] * (0.5 if m is a else 2.0))
    want = []
    for m in (a, b):
        m.step()
        torch.cuda.synchronize()
        want.append({k: v.clone() for k, v in m.o.items()})
        for v in m.o.values():
            v.fill_(float("nan"))
    graphs[0].replay()
    graphs[1].replay()
    fresh.step()
    graphs[0].replay()
    torch.cuda.synchronize()
    q.qffn_check_status()
    for m, w in zip((a, b), want):
        for k, v in w.items():
            assert torch.equal(m.o[k], v), k


def test_same_bits_every_run(q):
    """No result depends on the order in which blocks finish."""
    for M in (33, 333, 2100):
        b = Mlp(q, M, 520, 2056, seed=3)
        b.step()
        torch.cuda.synchronize()
        first = {k: v.clone() for k, v in b.o.items()}
        for _ in range(5):
            b.ws.fill_(0xA5)                           # whatever the workspace holds
            b.step()
        torch.cuda.synchronize()
        for k, v in first.items():
            assert torch.equal(b.o[k], v), (M, k)


def test_rows_behind_the_last_stay(q):
    """Outputs in larger buffers: what lies behind the last row is left as it was."""
    C, H = 264, 520
    for M in (1, 33, 129, 300):
        big = torch.full((M + 300, H), 7.0, dtype=bf16, device="cuda")
        x, w, w1 = _t(1, M, C).cuda(), _t(2, H, C).cuda(), _t(3, 2 * H, C).cuda()
        q.qffn_linear(big, None, x, w, None, None, q.QFFN_ACT_RELU, M, H, C, _ws(q.qffn_linear_workspace_size(M, H, C)))
        q.qffn_gated_linear(big, x, w1, q.QFFN_ACT_SILU, M, C, H, _ws(q.qffn_gated_linear_workspace_size(M, C, H)))
        q.qffn_check_status()
        assert (big[M:] == 7.0).all() and torch.isfinite(big[:M].float()).all()
