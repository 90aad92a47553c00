"""The operators around the bf16 feed-forward blocks, and the cases they are measured on.

Layer norm and its gradient, the gradient of the RMS norm, the matrix product with bias, activation and residual and
its gradient, and the gated pair of projections and its gradient.  ``run`` computes a case with elementary torch
operations in 32 bits, or, where ``own`` is true, with the calls of this repository's package.  ``exact`` gives the
same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "gelu", "gelu_tanh", "silu")
EPS = 1e-5


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one generated token's norm: the call's latency
        dict(name="layernorm_token", op="layernorm", rows=1, cols=4096, residual=False),
        # the residual sum and norm of a batch of four sequences of 2048 tokens
        dict(name="layernorm_batch", op="layernorm", rows=8192, cols=4096, residual=True),
        # the same layer's gradient in a training step of eight such sequences
        dict(name="layernorm_grad_batch", op="layernorm_backward", rows=16384, cols=4096, dres=True),
        # the RMS norm's gradient for a short, odd number of tokens (fine-tuning on single texts)
        dict(name="rmsnorm_grad_short", op="rmsnorm_backward", rows=77, cols=2048, dres=True),
        # the RMS norm's gradient in the training step of the FP8 block
        dict(name="rmsnorm_grad_batch", op="rmsnorm_backward", rows=16384, cols=4096, dres=True),
        # one generated token's down projection, added to the residual stream
        dict(name="linear_token", op="linear", rows=1, cols=4096, inner=14336, act="none", bias=False, residual=True, save_z=False),
        # the first projection of an ungated block for a batch of short prompts, kept for its gradient
        dict(name="linear_gelu_prompts", op="linear", rows=333, cols=8192, inner=2048, act="gelu", bias=True, residual=False, save_z=True),
        # the FP8 down projection of a prefill, its residual sum fused
        dict(name="linear_fp8_prefill", op="linear_fp8", rows=8192, cols=4096, inner=14336, act="none", bias=True, residual=True, save_z=False),
        # that projection's gradients in a training step
        dict(name="linear_grad_batch", op="linear_backward", rows=4096, cols=8192, inner=2048, act="gelu", bias=True, accumulate=False),
        # one generated token's gate and up projections
        dict(name="gated_token", op="gated", rows=1, cols=14336, inner=4096, act="silu"),
        # gate and up projections of a prefill of four sequences of 2048 tokens
        dict(name="gated_prefill", op="gated", rows=8192, cols=14336, inner=4096, act="silu"),
        # the gated pair's gradients, weight gradients summed over micro-batches
        dict(name="gated_grad_batch", op="gated_backward", rows=2048, cols=8192, inner=2048, act="silu", accumulate=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["layernorm", "layernorm_backward", "rmsnorm_backward", "linear", "linear", "linear_fp8",
                     "linear_backward", "gated", "gated_backward"])
    if "norm" in op:
        cols = 8 * _log(rng, 8, 2048)                               # 64 to 16384
        rows = _log(rng, 1, max(1, min(16384, 16384 * 4096 // cols)))
        case = dict(op=op, rows=rows, cols=cols)
        case["residual" if op == "layernorm" else "dres"] = rng.random() < 0.6
        return case
    step = 16 if op == "linear_fp8" else 8
    cols, inner = 8 * _log(rng, 16, 1792), step * _log(rng, 128 // step, 14336 // step)
    passes = {"linear": 1, "linear_fp8": 1, "linear_backward": 2, "gated": 2, "gated_backward": 6}[op]
    budget = (1 << 39) // (cols * inner * passes)                   # at most the prefill's products
    case = dict(op=op, rows=_log(rng, 1, max(1, min(8192, budget))), cols=cols, inner=inner)
    if op in ("linear", "linear_fp8"):
        case.update(act=rng.choice(ACTS), bias=rng.random() < 0.5, residual=rng.random() < 0.5, save_z=rng.random() < 0.3)
    elif op == "linear_backward":
        case.update(act=rng.choice(ACTS), bias=rng.random() < 0.7, accumulate=rng.random() < 0.4)
    else:
        case.update(act=rng.choice(ACTS[1:]))
        if op == "gated_backward":
            case.update(accumulate=rng.random() < 0.4)
    return case


# ------------------------------------------------------------------------------------------------ inputs

def _normal(gen, shape, std, mean=0.0):
    t = torch.empty(shape, dtype=torch.float32, device="cuda").normal_(mean, std, generator=gen)
    return t.to(torch.bfloat16)


def _stream(gen, rows, cols):
    """Hidden states as a residual stream has them: rows of different size and offset, a few channels far out."""
    t = torch.empty((rows, cols), dtype=torch.float32, device="cuda").normal_(0.0, 1.0, generator=gen)
    t *= torch.empty((rows, 1), dtype=torch.float32, device="cuda").uniform_(0.5, 2.0, generator=gen)
    t += torch.empty((rows, 1), dtype=torch.float32, device="cuda").normal_(0.0, 0.3, generator=gen)
    t[:, 3::251] *= 8.0
    return t.to(torch.bfloat16)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, rows, cols = case["op"], case["rows"], case["cols"]
    s = dict(case)
    if "norm" in op:
        s["gain"] = _normal(gen, (cols,), 0.1, 1.0)
        if op == "layernorm":
            s["x"] = _stream(gen, rows, cols)
            s["shift"] = _normal(gen, (cols,), 0.1)
            s["res"] = _stream(gen, rows, cols) if case["residual"] else None
        else:
            s["r"] = _stream(gen, rows, cols)
            s["dy"] = _normal(gen, (rows, cols), 1e-2)
            s["dr"] = _normal(gen, (rows, cols), 1e-2) if case["dres"] else None
            r = s["r"].float()
            s["mean"] = r.mean(1) if op == "layernorm_backward" else None
            mid = r - s["mean"][:, None] if op == "layernorm_backward" else r
            s["rstd"] = (mid.square().mean(1) + EPS).rsqrt()
        return s
    inner = case["inner"]
    wrows = 2 * cols if op.startswith("gated") else cols
    s["w"] = _normal(gen, (wrows, inner), 0.02)
    if op == "linear_fp8":
        # E4M3 records of the activations and the weights, each with its scale
        for name, t in (("x", _normal(gen, (rows, inner), 1.0)), ("w", s["w"])):
            amax = t.float().abs().max()
            s[name] = (t.float() * (448.0 / amax)).to(torch.float8_e4m3fn)
            s[name + "_scale"] = (amax / 448.0).reshape(1)
    else:
        s["x"] = _normal(gen, (rows, inner), 1.0)
    if op in ("linear", "linear_fp8"):
        s["b"] = _normal(gen, (cols,), 0.1) if case["bias"] else None
        s["res"] = _stream(gen, rows, cols) if case["residual"] else None
    else:
        s["dout"] = _normal(gen, (rows, cols), 1e-3)
        if op == "linear_backward":
            s["z"] = _normal(gen, (rows, cols), 1.2)
        if op in ("linear_backward", "gated_backward"):
            s["dw"] = _normal(gen, (wrows, inner), 1e-3) if case["accumulate"] else None
    return s


# ------------------------------------------------------------------------------------------------ plain forms

def _act(z, act):
    if act == "relu":
        return z.clamp_min(0)
    if act == "gelu":
        return z * 0.5 * torch.erfc(z * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "gelu":
        return 0.5 * torch.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if act == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        p = torch.sigmoid(c * (z + 0.044715 * z * z * z))
        return p + z * p * (1 - p) * c * (1 + 3 * 0.044715 * z * z)
    if act == "silu":
        p = torch.sigmoid(z)
        return p * (1 + z * (1 - p))
    return torch.ones_like(z)


def _plain(s):
    op, bf = s["op"], torch.bfloat16
    if op == "layernorm":
        r = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(bf)
        f = r.float()
        mean = f.mean(1, keepdim=True)
        mid = f - mean
        rstd = (mid.square().mean(1, keepdim=True) + EPS).rsqrt()
        y = (mid * rstd * s["gain"].float() + s["shift"].float()).to(bf)
        return dict(y=y, mean=mean[:, 0], rstd=rstd[:, 0], r=None if s["res"] is None else r)
    if op in ("layernorm_backward", "rmsnorm_backward"):
        centred = op == "layernorm_backward"
        r, dy, rstd = s["r"].float(), s["dy"].float(), s["rstd"][:, None]
        hat = (r - s["mean"][:, None]) * rstd if centred else r * rstd
        g = dy * s["gain"].float()
        dx = g - hat * (g * hat).mean(1, keepdim=True)
        if centred:
            dx = dx - g.mean(1, keepdim=True)
        dx = dx * rstd
        if s["dr"] is not None:
            dx = dx + s["dr"].float()
        return dict(dx=dx.to(bf), dgain=(dy * hat).sum(0), dshift=dy.sum(0) if centred else None)
    x, w = s["x"].float(), s["w"].float()
    if op in ("linear", "linear_fp8"):
        z = x @ w.t()
        if op == "linear_fp8":
            z = z * (s["x_scale"] * s["w_scale"])
        if s["b"] is not None:
            z = z + s["b"].float()
        out = _act(z, s["act"])
        if s["res"] is not None:
            out = out + s["res"].float()
        return dict(out=out.to(bf), z=z.to(bf) if s["save_z"] else None)
    if op == "gated":
        return dict(h=(_act(x @ w[:s["cols"]].t(), s["act"]) * (x @ w[s["cols"]:].t())).to(bf))
    if op == "linear_backward":
        dz = s["dout"].float() * _act_grad(s["z"].float(), s["act"])
    else:
        gate, up, dh = x @ w[:s["cols"]].t(), x @ w[s["cols"]:].t(), s["dout"].float()
        dz = torch.cat([dh * up * _act_grad(gate, s["act"]), dh * _act(gate, s["act"])], 1)
    dw = dz.t() @ x
    if s["dw"] is not None:
        dw = dw + s["dw"].float()
    out = dict(dx=(dz @ w).to(bf), dw=dw.to(bf))
    if s.get("bias"):
        out["db"] = dz.sum(0)
    return out


# ------------------------------------------------------------------------------------------------ the package's calls

def _buffers(q, s):
    """Outputs and workspace, which a program keeps from step to step."""
    op, rows, cols = s["op"], s["rows"], s["cols"]

    def new(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="cuda")

    f32 = torch.float32
    if op == "layernorm":
        return dict(y=new(rows, cols), mean=new(rows, dtype=f32), rstd=new(rows, dtype=f32),
                    r=new(rows, cols) if s["res"] is not None else None)
    if "norm" in op:
        b = dict(dx=new(rows, cols), dgain=new(cols, dtype=f32), dshift=new(cols, dtype=f32) if op == "layernorm_backward" else None)
        size = q.qffn_norm_backward_workspace_size(rows, cols)
    elif op in ("linear", "linear_fp8"):
        b = dict(out=new(rows, cols), z=new(rows, cols) if s["save_z"] else None)
        size = (q.qffn_linear_workspace_size if op == "linear" else q.qffn_linear_fp8_workspace_size)(rows, cols, s["inner"])
    elif op == "gated":
        b = dict(h=new(rows, cols))
        size = q.qffn_gated_linear_workspace_size(rows, s["inner"], cols)
    else:
        b = dict(dx=new(rows, s["inner"]), dw=new(*s["w"].shape))
        if op == "linear_backward":
            b["db"] = new(cols, dtype=f32) if s["bias"] else None
            size = q.qffn_linear_backward_workspace_size(rows, cols, s["inner"])
        else:
            size = q.qffn_gated_linear_backward_workspace_size(rows, s["inner"], cols)
    s["ws"] = new(size, dtype=torch.uint8)
    return b


def _own(s):
    import transformer_ffn_block_gb300 as q
    b = s.get("buffers")
    if b is None:
        b = s["buffers"] = _buffers(q, s)
    op, rows, cols = s["op"], s["rows"], s["cols"]
    if op == "layernorm":
        q.qffn_layernorm_absmax(b["r"], b["y"], b["mean"], b["rstd"], None, s["res"], s["x"], s["gain"], s["shift"], EPS, rows, cols)
        return b
    if op == "layernorm_backward":
        q.qffn_layernorm_backward(b["dx"], b["dgain"], b["dshift"], None, s["dy"], s["dr"], s["r"], s["mean"], s["rstd"],
                                  s["gain"], rows, cols, False, s["ws"])
        return b
    if op == "rmsnorm_backward":
        q.qffn_rmsnorm_backward(b["dx"], b["dgain"], None, s["dy"], s["dr"], s["r"], s["rstd"], s["gain"], rows, cols, False, s["ws"])
        return b
    inner, act = s["inner"], getattr(q, "QFFN_ACT_" + s["act"].upper())
    if op == "linear":
        q.qffn_linear(b["out"], b["z"], s["x"], s["w"], s["b"], s["res"], act, rows, cols, inner, s["ws"])
        return b
    if op == "linear_fp8":
        q.qffn_linear_fp8(b["out"], b["z"], s["x"], s["x_scale"], s["w"], s["w_scale"], s["b"], s["res"], act, rows, cols, inner, s["ws"])
        return b
    if op == "gated":
        q.qffn_gated_linear(b["h"], s["x"], s["w"], act, rows, inner, cols, s["ws"])
        return b
    if s["dw"] is not None:
        b["dw"].copy_(s["dw"])                                      # what the micro-batches before this one left
        if b.get("db") is not None:
            b["db"].zero_()                                         # (they left no bias gradient)
    if op == "linear_backward":
        q.qffn_linear_backward(b["dx"], b["dw"], b["db"], s["dout"], s["z"], s["x"], s["w"], act, rows, cols, inner,
                               s["dw"] is not None, s["ws"])
    else:
        q.qffn_gated_linear_backward(b["dx"], b["dw"], s["dout"], s["x"], s["w"], act, rows, inner, cols, s["dw"] is not None, s["ws"])
    return b


def run(s):
    if own:
        return _own(s)
    return _plain(s)


# ------------------------------------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op, rows, cols = case["op"], case["rows"], case["cols"]
    n = rows * cols
    if op == "layernorm":
        return dict(bytes=n * (8 if case["residual"] else 4) + 8 * rows + 4 * cols, flops=8 * n)
    if "norm" in op:
        return dict(bytes=n * (8 if case["dres"] else 6) + 8 * rows + 10 * cols, flops=14 * n)
    inner = case["inner"]
    if op in ("linear", "linear_fp8"):
        size = 1 if op == "linear_fp8" else 2
        return dict(bytes=(rows + cols) * inner * size + 2 * n * (1 + case["residual"] + case["save_z"]) + 2 * cols * case["bias"],
                    flops=2 * n * inner)
    if op == "gated":
        return dict(bytes=2 * (rows * inner + 2 * cols * inner + n), flops=4 * n * inner)
    if op == "linear_backward":
        return dict(bytes=2 * (n * (1 if case["act"] == "none" else 2) + 2 * rows * inner + cols * inner * (3 if case["accumulate"] else 2))
                    + 4 * cols * case["bias"], flops=4 * n * inner)
    return dict(bytes=2 * (n + 2 * rows * inner + 2 * cols * inner * (3 if case["accumulate"] else 2)), flops=12 * n * inner)


# ------------------------------------------------------------------------------------------------ the definitions in 64 bits

def _normal_cdf(v):
    return torch.special.erfc(-v / 2.0 ** 0.5) / 2


def _phi_and_slope(v, act):
    """phi(v) and its derivative, in 64 bits."""
    if act == "none":
        return v, torch.ones_like(v)
    if act == "relu":
        return torch.where(v > 0, v, torch.zeros_like(v)), torch.where(v > 0, torch.ones_like(v), torch.zeros_like(v))
    if act == "silu":
        sig = 1 / (1 + torch.exp(-v))
        return v * sig, sig + v * sig * torch.exp(-v) * sig
    if act == "gelu":
        return v * _normal_cdf(v), _normal_cdf(v) + v * torch.exp(-v * v / 2) / (2 * math.pi) ** 0.5
    t = torch.tanh((2 / math.pi) ** 0.5 * (v + 0.044715 * v ** 3))
    dt = (1 - t * t) * (2 / math.pi) ** 0.5 * (1 + 0.134145 * v * v)
    return v * (1 + t) / 2, (1 + t) / 2 + v * dt / 2


def exact(case, seed):
    s = prepare(case, seed)
    d = {k: v.to(torch.float64) for k, v in s.items() if isinstance(v, torch.Tensor)}
    op, cols = case["op"], case["cols"]
    if op == "layernorm":
        r = d["x"]
        if case["residual"]:
            r = (d["x"] + d["res"]).to(torch.bfloat16).to(torch.float64)   # the residual stream is kept in bf16
        var, mean = torch.var_mean(r, dim=1, correction=0)
        rstd = 1 / torch.sqrt(var + EPS)
        y = (r - mean.unsqueeze(1)) * rstd.unsqueeze(1) * d["gain"] + d["shift"]
        return dict(y=y, mean=mean, rstd=rstd, r=r if case["residual"] else None)
    if "norm" in op:
        # x-hat is r shifted and scaled by the row's statistics; dx is the gradient through both statistics
        mean = d["mean"].unsqueeze(1) if "mean" in d else torch.zeros_like(d["rstd"]).unsqueeze(1)
        xhat = (d["r"] - mean) * d["rstd"].unsqueeze(1)
        up = d["dy"] * d["gain"]
        along = torch.einsum("nc,nc->n", up, xhat).unsqueeze(1) / cols
        level = up.sum(1, keepdim=True) / cols if "mean" in d else 0.0
        dx = (up - level - along * xhat) * d["rstd"].unsqueeze(1)
        if case["dres"]:
            dx = dx + d["dr"]
        return dict(dx=dx, dgain=torch.einsum("nc,nc->c", d["dy"], xhat), dshift=d["dy"].sum(0) if "mean" in d else None)
    x, w = d["x"], d["w"]
    if op in ("linear", "linear_fp8"):
        v = torch.einsum("mk,nk->mn", x, w)
        if op == "linear_fp8":
            v = v * d["x_scale"] * d["w_scale"]
        if case["bias"]:
            v = v + d["b"]
        out = _phi_and_slope(v, case["act"])[0]
        return dict(out=out + d["res"] if case["residual"] else out, z=v if case["save_z"] else None)
    if op == "linear_backward":
        dv = d["dout"] * _phi_and_slope(d["z"], case["act"])[1]
    else:
        pair = torch.einsum("mk,nk->mn", x, w)
        value, slope = _phi_and_slope(pair[:, :cols], case["act"])
        if op == "gated":
            return dict(h=value * pair[:, cols:])
        dv = torch.cat((d["dout"] * pair[:, cols:] * slope, d["dout"] * value), dim=1)
    out = dict(dx=torch.einsum("mn,nk->mk", dv, w), dw=torch.einsum("mn,mk->nk", dv, x))
    if case["accumulate"]:
        out["dw"] = out["dw"] + d["dw"]
    if case.get("bias"):
        out["db"] = dv.sum(0)
    return out
