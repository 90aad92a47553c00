"""Block-scaled FP8 and grouped products beside the feed-forward block, and the cases they are measured on.

The RMS norm and SwiGLU with an E4M3 output and a scale for each 128 values of a row, the E4M3 product with such scales
(weights: one per 128 x 128), and the products of several experts' ragged groups of rows, in bf16 with their gradients and in
E4M3 with scales.  ``run`` computes a case with elementary torch operations in 32 bits, or, where ``own`` is true, with
the calls of this repository's package.  ``exact`` gives the same outputs from the definitions in 64 bits.
"""
import math

import torch

own = False

EPS = 1e-5
E4M3, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one generated token's residual sum and norm, quantised for the projection behind it: the call's latency
        dict(name="rmsnorm_blocks_token", op="rmsnorm_blocks", rows=1, cols=4096, residual=True),
        # the same for a prefill of four sequences of 2048 tokens
        dict(name="rmsnorm_blocks_batch", op="rmsnorm_blocks", rows=8192, cols=4096, residual=True),
        # the SwiGLU between two expert products in a decode step of a small batch (an odd number of routed rows)
        dict(name="swiglu_blocks_decode", op="swiglu_blocks", rows=37, cols=2048),
        # the SwiGLU of a prefill
        dict(name="swiglu_blocks_batch", op="swiglu_blocks", rows=8192, cols=14336),
        # one generated token's down projection, added to the residual stream
        dict(name="linear_blocks_token", op="linear_blocks", rows=1, cols=4096, inner=14336, bias=False, residual=True),
        # the down projection of a prefill, added to the residual stream
        dict(name="linear_blocks_prefill", op="linear_blocks", rows=8192, cols=4096, inner=14336, bias=False, residual=True),
        # one generated token sent to two of eight experts: their gate and up projections
        dict(name="grouped_token", op="grouped", tokens=1, top=2, experts=8, spare=0, cols=28672, inner=4096),
        # many small experts in a forward pass of short sequences
        dict(name="grouped_batch", op="grouped", tokens=1024, top=8, experts=64, spare=0, cols=2048, inner=2048),
        # gradients of a fine-tuning step on a single text of odd length in a padded buffer, summed over micro-batches
        dict(name="grouped_grad_short", op="grouped_backward", tokens=389, top=2, experts=16, spare=22, cols=2048, inner=1032,
             accumulate=True),
        # gradients of a training step of 8192 tokens
        dict(name="grouped_grad_batch", op="grouped_backward", tokens=8192, top=2, experts=8, spare=0, cols=4096, inner=2048,
             accumulate=False),
        # a decode step of a batch of 32 sequences over many small experts
        dict(name="grouped_blocks_decode", op="grouped_blocks", tokens=32, top=8, experts=64, spare=0, cols=4096, inner=2048),
        # gate and up projections of a prefill over eight large experts
        dict(name="grouped_blocks_prefill", op="grouped_blocks", tokens=4096, top=2, experts=8, spare=0, cols=28672, inner=4096),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rmsnorm_blocks", "swiglu_blocks", "linear_blocks", "linear_blocks", "grouped", "grouped_backward",
                     "grouped_blocks", "grouped_blocks"])
    if op in ("rmsnorm_blocks", "swiglu_blocks"):
        cols = 16 * _log(rng, 4, 1024 if op == "rmsnorm_blocks" else 896)      # 64 to 16384 or 14336
        rows = _log(rng, 1, max(1, min(16384, 8192 * (4096 if op == "rmsnorm_blocks" else 14336) // cols)))
        case = dict(op=op, rows=rows, cols=cols)
        if op == "rmsnorm_blocks":
            case["residual"] = rng.random() < 0.6
        return case
    step = 8 if op in ("grouped", "grouped_backward") else 16
    inner = step * _log(rng, 128 // step, 14336 // step)
    cols = 8 * _log(rng, 16, 1792)
    if op == "linear_blocks":
        rows = _log(rng, 1, max(1, min(8192, (1 << 39) // (cols * inner))))
        return dict(op=op, rows=rows, cols=cols, inner=inner, bias=rng.random() < 0.4, residual=rng.random() < 0.5)
    # at most the large experts' weights and the prefill's products
    experts = _log(rng, 1, max(1, min(128, (28672 * 4096 * 8) // (cols * inner))))
    top = min(experts, rng.choice([1, 2, 4, 8]))
    passes = 2 if op == "grouped_backward" else 1
    tokens = _log(rng, 1, max(1, min(8192, (1 << 39) // (cols * inner * passes * top))))
    case = dict(op=op, tokens=tokens, top=top, experts=experts, spare=rng.choice([0, 0, 1, 19]), cols=cols, inner=inner)
    if op == "grouped_backward":
        case["accumulate"] = rng.random() < 0.4
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


def _records(t, by):
    """E4M3 codes and E8M0 scales of ``t`` [..., rows, cols] for blocks of ``by`` rows x 128 columns."""
    *lead, rows, cols = t.shape
    br, bc = -(-rows // by), -(-cols // 128)
    padded = torch.nn.functional.pad(t.float(), (0, bc * 128 - cols, 0, br * by - rows))
    blocks = padded.view(*lead, br, by, bc, 128)
    code = _scale_code(blocks.abs().amax((-3, -1)))
    q = blocks * _power(127 - code)[..., :, None, :, None]
    return q.view(*lead, br * by, bc * 128)[..., :rows, :cols].to(E4M3).contiguous(), code.to(torch.uint8).view(E8M0)


def _offsets(case, seed):
    """Routed rows by expert: each token goes to its ``top`` best of scores with a preference, so some experts get many."""
    gen = torch.Generator().manual_seed(seed)
    scores = torch.randn(case["tokens"], case["experts"], generator=gen) + 0.7 * torch.randn(case["experts"], generator=gen)
    sizes = torch.bincount(scores.topk(case["top"], dim=1).indices.flatten(), minlength=case["experts"])
    return torch.cat([torch.zeros(1, dtype=torch.int64), sizes.cumsum(0)]), int(sizes.max())


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, cols = case["op"], case["cols"]
    s = dict(case)
    if op == "rmsnorm_blocks":
        s["gain"] = _normal(gen, (cols,), 0.1, 1.0)
        s["x"] = _stream(gen, case["rows"], cols)
        s["res"] = _stream(gen, case["rows"], cols) if case["residual"] else None
        return s
    if op == "swiglu_blocks":
        s["gate_up"] = _normal(gen, (case["rows"], 2 * cols), 1.2)
        return s
    inner = case["inner"]
    if op == "linear_blocks":
        s["x"], s["x_scale"] = _records(_stream(gen, case["rows"], inner), 1)
        s["w"], s["w_scale"] = _records(_normal(gen, (cols, inner), 0.02), 128)
        s["b"] = _normal(gen, (cols,), 0.1) if case["bias"] else None
        s["res"] = _stream(gen, case["rows"], cols) if case["residual"] else None
        return s
    offsets, s["most"] = _offsets(case, seed)
    s["rows"] = rows = case["tokens"] * case["top"] + case["spare"]
    s["offsets"] = offsets.to(torch.int32).cuda()
    # row -> its expert and its place there, for the plain form
    routed = torch.arange(int(offsets[-1]))
    s["expert"] = torch.searchsorted(offsets[1:], routed, right=True)
    s["place"] = (routed - offsets[s["expert"]]).cuda()
    s["expert"] = s["expert"].cuda()
    w = _normal(gen, (case["experts"], cols, inner), 0.02)
    if op == "grouped_blocks":
        s["w"], s["w_scale"] = _records(w, 128)
        s["x"], s["x_scale"] = _records(_stream(gen, rows, inner), 1)
    else:
        s["w"], s["x"] = w, _normal(gen, (rows, inner), 1.0)
    if op == "grouped_backward":
        s["dout"] = _normal(gen, (rows, cols), 1e-3)
        s["dw"] = _normal(gen, w.shape, 1e-3) if case["accumulate"] else None
    return s


# ------------------------------------------------------------------------------------------------ plain forms

def _power(e):
    """2 ** e for whole numbers, exactly."""
    return torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)


def _scale_code(amax):
    """The E8M0 code of the smallest power of two times 448 (1.75 * 2 ** 8) that holds amax; 127 for zero."""
    mantissa, e = torch.frexp(amax)                                   # amax = mantissa * 2 ** e, mantissa in [0.5, 1)
    code = (e - 9 + (mantissa > 0.875).to(e.dtype) + 127).clamp_min(0)
    return torch.where(amax > 0, code, torch.full_like(code, 127))


def _to_blocks(v):
    """E4M3 values and scales of the rows of v (32 bits)."""
    rows, cols = v.shape
    n = -(-cols // 128)
    blocks = torch.nn.functional.pad(v, (0, n * 128 - cols)).view(rows, n, 128)
    code = _scale_code(blocks.abs().amax(2))
    q = (blocks * _power(127 - code)[..., None]).view(rows, n * 128)[:, :cols]
    return dict(q=q.to(E4M3), scale=code.to(torch.uint8).view(E8M0))


def _values(q, scale, by):
    """What codes [..., rows, cols] with scales for ``by`` x 128 of them stand for, in 32 bits."""
    rows, cols = q.shape[-2:]
    full = scale.float().repeat_interleave(128, -1)[..., :cols]
    if by > 1:
        full = full.repeat_interleave(by, -2)[..., :rows, :]
    return q.float() * full


def _spread(s, t):
    """Rows [routed, n] as [experts, most, n], zeros where an expert has fewer."""
    padded = torch.zeros((s["experts"], s["most"], t.shape[1]), dtype=torch.float32, device=t.device)
    padded[s["expert"], s["place"]] = t[:len(s["place"])].float()
    return padded


def _gather(s, padded):
    """The reverse, in bf16; rows behind the last group are zero."""
    out = torch.zeros((s["rows"], padded.shape[2]), dtype=torch.bfloat16, device=padded.device)
    out[:len(s["place"])] = padded[s["expert"], s["place"]].to(torch.bfloat16)
    return out


def _plain(s):
    op, bf = s["op"], torch.bfloat16
    if op == "rmsnorm_blocks":
        r = s["x"] if s["res"] is None else (s["x"].float() + s["res"].float()).to(bf)
        f = r.float()
        rstd = (f.square().mean(1, keepdim=True) + EPS).rsqrt()
        return dict(**_to_blocks(f * rstd * s["gain"].float()), rstd=rstd[:, 0], r=None if s["res"] is None else r)
    if op == "swiglu_blocks":
        g, u = s["gate_up"][:, :s["cols"]].float(), s["gate_up"][:, s["cols"]:].float()
        return _to_blocks(g * torch.sigmoid(g) * u)
    if op == "linear_blocks":
        out = _values(s["x"], s["x_scale"], 1) @ _values(s["w"], s["w_scale"], 128).t()
        if s["b"] is not None:
            out = out + s["b"].float()
        if s["res"] is not None:
            out = out + s["res"].float()
        return dict(out=out.to(bf))
    if op == "grouped_blocks":
        x, w = _values(s["x"], s["x_scale"], 1), _values(s["w"], s["w_scale"], 128)
    else:
        x, w = s["x"], s["w"].float()
    x = _spread(s, x)
    if op != "grouped_backward":
        return dict(out=_gather(s, torch.bmm(x, w.transpose(1, 2))))
    dout = _spread(s, s["dout"])
    dw = torch.bmm(dout.transpose(1, 2), x)
    if s["dw"] is not None:
        dw = dw + s["dw"].float()
    return dict(dx=_gather(s, torch.bmm(dout, w)), dw=dw.to(bf))


# ------------------------------------------------------------------------------------------------ the package's calls

def _buffers(s):
    """Outputs, which a program keeps from step to step."""
    op, rows, cols = s["op"], s["rows"], s["cols"]

    def new(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    if op in ("rmsnorm_blocks", "swiglu_blocks"):
        b = dict(q=new(rows, cols, dtype=torch.uint8).view(E4M3), scale=new(rows, -(-cols // 128), dtype=torch.uint8).view(E8M0))
        if op == "rmsnorm_blocks":
            b.update(rstd=new(rows, dtype=torch.float32), r=new(rows, cols) if s["res"] is not None else None)
        return b
    if op == "grouped_backward":
        return dict(dx=new(rows, s["inner"]), dw=new(*s["w"].shape))
    return dict(out=new(rows, cols))


def _own(s):
    import transformer_ffn_block_gb300 as q
    b = s.get("buffers")
    if b is None:
        b = s["buffers"] = _buffers(s)
    op, rows, cols = s["op"], s["rows"], s["cols"]
    if op == "rmsnorm_blocks":
        q.qffn_rmsnorm_quantize_blocks(b["r"], None, b["q"], b["scale"], b["rstd"], s["res"], s["x"], s["gain"], EPS, rows, cols)
    elif op == "swiglu_blocks":
        q.qffn_swiglu_quantize_blocks(None, b["q"], b["scale"], s["gate_up"], rows, cols)
    elif op == "linear_blocks":
        q.qffn_linear_fp8_blocks(b["out"], s["x"], s["x_scale"], s["w"], s["w_scale"], s["b"], s["res"], rows, cols, s["inner"])
    elif op == "grouped":
        q.qffn_grouped_linear(b["out"], s["x"], s["w"], s["offsets"], s["experts"], rows, cols, s["inner"])
    elif op == "grouped_blocks":
        q.qffn_grouped_linear_fp8_blocks(b["out"], s["x"], s["x_scale"], s["w"], s["w_scale"], s["offsets"], s["experts"], rows, cols,
                                         s["inner"])
    else:
        if s["dw"] is not None:
            b["dw"].copy_(s["dw"])                                    # what the micro-batches before this one left
        q.qffn_grouped_linear_backward(b["dx"], b["dw"], s["dout"], s["x"], s["w"], s["offsets"], s["experts"], rows, cols, s["inner"],
                                       s["dw"] is not None)
    return b


def run(s):
    if own:
        return _own(s)
    return _plain(s)


# ------------------------------------------------------------------------------------------------ what a pass cannot do without

def work(case):
    op, cols = case["op"], case["cols"]
    if op == "rmsnorm_blocks":
        n = case["rows"] * cols
        return dict(bytes=n * (7 if case["residual"] else 3) + n // 128 + 4 * case["rows"] + 2 * cols, flops=8 * n)
    if op == "swiglu_blocks":
        n = case["rows"] * cols
        return dict(bytes=5 * n + n // 128, flops=10 * n)
    inner = case["inner"]
    if op == "linear_blocks":
        rows = case["rows"]
        n = rows * cols
        return dict(bytes=(rows + cols) * inner + rows * inner // 128 + 2 * n * (1 + case["residual"]) + 2 * cols * case["bias"],
                    flops=2 * n * inner)
    rows, experts = case["tokens"] * case["top"], case["experts"]
    # experts that get a row at all, if none were preferred
    busy = experts * (1 - (1 - case["top"] / experts) ** case["tokens"])
    size = 1 if op == "grouped_blocks" else 2
    if op != "grouped_backward":
        return dict(bytes=int((rows + busy * cols) * inner * size + 2 * rows * cols), flops=2 * rows * cols * inner)
    # (dw of an expert without rows is written too)
    return dict(bytes=int(2 * (rows * cols + 2 * rows * inner + (busy + experts * (2 if case["accumulate"] else 1)) * cols * inner)),
                flops=4 * rows * cols * inner)


# ------------------------------------------------------------------------------------------------ the definitions in 64 bits

def _e4m3(v):
    """v rounded to the nearest value of three fraction bits, exponent -6 at least (ties to even)."""
    e = torch.floor(torch.log2(v.abs().clamp_min(2.0 ** -20))).clamp_min(-6)
    step = 2.0 ** (e - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _blocks_exactly(v):
    q, scale = torch.zeros_like(v), []
    for at in range(0, v.shape[1], 128):
        part = v[:, at:at + 128]
        top = part.abs().max(dim=1, keepdim=True).values
        s = torch.where(top > 0, 2.0 ** torch.ceil(torch.log2(top / 448)).clamp_min(-127), torch.ones_like(top))
        q[:, at:at + 128] = _e4m3(part / s)
        scale.append(s)
    return dict(q=q, scale=torch.cat(scale, 1))


def _decoded(q, scale, by):
    """Codes and scales as 64-bit values, block column by block column."""
    v = q.to(torch.float32).to(torch.float64)
    s = scale.to(torch.float32).to(torch.float64)
    for j in range(s.shape[-1]):
        rows = s[..., j]
        if by > 1:
            rows = rows.repeat_interleave(by, dim=-1)[..., :v.shape[-2]]
        v[..., 128 * j:128 * (j + 1)] *= rows.unsqueeze(-1)
    return v


def exact(case, seed):
    s = prepare(case, seed)
    op, cols = case["op"], case["cols"]
    if op == "rmsnorm_blocks":
        r = s["x"].double()
        if case["residual"]:
            r = (r + s["res"].double()).to(torch.bfloat16).double()       # the residual stream is kept in bf16
        rstd = 1 / torch.sqrt((r * r).sum(1) / cols + EPS)
        return dict(**_blocks_exactly(r * rstd.unsqueeze(1) * s["gain"].double()), rstd=rstd, r=r if case["residual"] else None)
    if op == "swiglu_blocks":
        g, u = s["gate_up"].double().chunk(2, dim=1)
        return _blocks_exactly(g / (1 + torch.exp(-g)) * u)
    if op == "linear_blocks":
        out = torch.einsum("mk,nk->mn", _decoded(s["x"], s["x_scale"], 1), _decoded(s["w"], s["w_scale"], 128))
        if case["bias"]:
            out += s["b"].double()
        if case["residual"]:
            out += s["res"].double()
        return dict(out=out)
    ends = s["offsets"].tolist()
    x = _decoded(s["x"], s["x_scale"], 1) if op == "grouped_blocks" else s["x"].double()
    out = torch.zeros((s["rows"], case["inner"] if op == "grouped_backward" else cols), dtype=torch.float64, device="cuda")
    dw = torch.zeros(s["w"].shape, dtype=torch.float64, device="cuda") if op == "grouped_backward" else None
    for g in range(case["experts"]):
        lo, hi = ends[g], ends[g + 1]
        if op == "grouped_backward":
            d = s["dout"][lo:hi].double()
            out[lo:hi] = d @ s["w"][g].double()
            dw[g] = d.t() @ x[lo:hi]
        elif hi > lo:
            w = _decoded(s["w"][g], s["w_scale"][g], 128) if op == "grouped_blocks" else s["w"][g].double()
            out[lo:hi] = x[lo:hi] @ w.t()
    if dw is None:
        return dict(out=out)
    if case["accumulate"]:
        dw += s["dw"].double()
    return dict(dx=out, dw=dw)
