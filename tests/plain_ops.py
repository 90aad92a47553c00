"""Plain 64-bit forms of the norm, linear and gated operators (torch float64 on the CPU), and the
error bounds their bf16 kernels are held to."""
import math

import torch

ACTS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}
HALF = 2.0 ** -8            # half a bf16 step, relative to the value
ACC = 2.0 ** -23            # one fp32 unit per added product (tensor-core sums are not specified as nearest)
ACT_REL = 2.0 ** -18        # fp32 activation: the exponential's argument and result, a quotient, a few products
SLOPE = 1.2                 # no activation here has a slope beyond this


def act(z, name):
    if name == "none":
        return z
    if name == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if name == "gelu":
        return z * 0.5 * torch.special.erfc(-z / math.sqrt(2.0))
    if name == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    return z / (1 + torch.exp(-z))


def act_grad(z, name):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        return 0.5 * torch.special.erfc(-z / math.sqrt(2.0)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        t = torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    s = 1 / (1 + torch.exp(-z))
    return s * (1 + z * (1 - s))


def layernorm(r, gain, shift, eps):
    mean = r.mean(1, keepdim=True)
    rstd = 1 / torch.sqrt(((r - mean) ** 2).mean(1, keepdim=True) + eps)
    y = (r - mean) * rstd * gain
    return (y if shift is None else y + shift), mean[:, 0], rstd[:, 0]


def norm_backward(dy, dres, r, mean, rstd, gain):
    """mean None: the RMS norm.  Returns dx, dgain, dshift and the bounds of dx and dgain."""
    mu = torch.zeros_like(rstd)[:, None] if mean is None else mean[:, None]
    rs = rstd[:, None]
    xh = (r - mu) * rs
    w = dy * gain
    c1 = (w * xh).mean(1, keepdim=True)
    c2 = w.mean(1, keepdim=True) if mean is not None else torch.zeros_like(c1)
    dx = rs * (w - c2 - xh * c1)
    if dres is not None:
        dx = dx + dres
    # xhat is off by the rounding of r - mean and of the product; the row sums by at most 32 fp32 steps
    d_xh = 2.0 ** -22 * (r.abs() + mu.abs()) * rs
    d_c1 = 2.0 ** -19 * (w * xh).abs().mean(1, keepdim=True) + (w.abs() * d_xh).mean(1, keepdim=True)
    d_c2 = 2.0 ** -19 * w.abs().mean(1, keepdim=True)
    b_dx = HALF * dx.abs() + rs * (c1.abs() * d_xh + xh.abs() * d_c1 + d_c2 + 2.0 ** -21 * (w.abs() + c2.abs() + (xh * c1).abs()))
    n = dy.shape[0]
    b_dg = (dy.abs() * d_xh).sum(0) + (n + 80) * 2.0 ** -24 * (dy * xh).abs().sum(0)
    b_ds = (n + 80) * 2.0 ** -24 * dy.abs().sum(0)
    return dx, (dy * xh).sum(0), dy.sum(0), b_dx, b_dg, b_ds


def linear(x, w, bias, residual, name, scale=1.0):
    """out, z and their bounds."""
    K = x.shape[1]
    z = scale * (x @ w.t())
    e = (K * ACC + 2.0 ** -21) * scale * (x.abs() @ w.abs().t())
    if bias is not None:
        z = z + bias
        e = e + 2.0 ** -23 * (z.abs() + bias.abs())
    a = act(z, name)
    out = a if residual is None else a + residual
    e_out = SLOPE * e + ACT_REL * a.abs() + 2.0 ** -23 * out.abs()
    return out, z, HALF * (out.abs() + e_out) + e_out, HALF * (z.abs() + e) + e


def products(dz, e_dz, x, w, old):
    """dx, dw of the (bf16-rounded) dz whose value before rounding is off by e_dz, and their bounds."""
    M, N = dz.shape
    e = HALF * (dz.abs() + e_dz) + e_dz
    dx, dw = dz @ w, dz.t() @ x
    big = dz.abs() + e
    b_dx = e @ w.abs() + (N * ACC + 2.0 ** -22) * (big @ w.abs())
    b_dw = e.t() @ x.abs() + (M * ACC + 2.0 ** -22) * (big.t() @ x.abs())
    if old is not None:
        dw = dw + old
        b_dw = b_dw + 2.0 ** -23 * dw.abs()
    return dx, dw, HALF * (dx.abs() + b_dx) + b_dx, HALF * (dw.abs() + b_dw) + b_dw


def linear_backward(dout, z, x, w, name, old=None):
    dz = dout if name == "none" else dout * act_grad(z, name)
    # act' is a sum of terms of size 1 at most, each to ACT_REL
    e = torch.zeros_like(dz) if name in ("none", "relu") else 4 * ACT_REL * dout.abs()
    dx, dw, b_dx, b_dw = products(dz, e, x, w, old)
    if name == "none":   # dz = dout is already bf16: no rounding of its own
        b_dx, b_dw = (HALF * v.abs() + 2 * (n * ACC + 2.0 ** -22) * a for v, n, a in
                      ((dx, dz.shape[1], dz.abs() @ w.abs()), (dw, dz.shape[0], dz.abs().t() @ x.abs())))
    b_db = e.sum(0) + (dz.shape[0] + 80) * 2.0 ** -24 * dz.abs().sum(0)
    return dx, dw, dz.sum(0), b_dx, b_dw, b_db


def gated(x, w1, name):
    H, K = w1.shape[0] // 2, x.shape[1]
    g, u = x @ w1[:H].t(), x @ w1[H:].t()
    eg = (K * ACC + 2.0 ** -22) * (x.abs() @ w1[:H].abs().t())
    eu = (K * ACC + 2.0 ** -22) * (x.abs() @ w1[H:].abs().t())
    a = act(g, name)
    ea = SLOPE * eg + ACT_REL * a.abs()
    h = a * u
    e = ea * (u.abs() + eu) + a.abs() * eu + 2.0 ** -23 * h.abs()
    return h, HALF * (h.abs() + e) + e, (g, u, a, eg, eu, ea)


def gated_backward(dh, x, w1, name, old=None):
    _, _, (g, u, a, eg, eu, ea) = gated(x, w1, name)
    s = act_grad(g, name)
    # no activation here has a second derivative beyond 1.2; relu' jumps where |g| is within its error
    es = 4 * ACT_REL + (SLOPE * eg if name != "relu" else (g.abs() <= eg).double())
    dz = torch.cat([dh * u * s, dh * a], 1)
    e = torch.cat([dh.abs() * (eu * s.abs() + (u.abs() + eu) * es), dh.abs() * ea], 1) + 2.0 ** -22 * dz.abs()
    dx, dw, b_dx, b_dw = products(dz, e, x, w1, old)
    return dz, HALF * (dz.abs() + e) + e, dx, dw, b_dx, b_dw


def check(got, want, bound, name):
    got = got.double().cpu()
    assert torch.isfinite(got).all(), f"{name}: not finite"
    err = (got - want).abs()
    worst = (err / bound.clamp_min(1e-300)).max().item() if err.numel() else 0.0
    assert bool((err <= bound + 1e-38).all()), f"{name}: {int((err > bound).sum())} of {err.numel()} beyond the bound, worst {worst:.3g}"
    return worst
