"""Calls whose every input was written by the call just before them, enqueued without a pause, give the bits
that the same calls give with a synchronisation behind each: nothing of the run before is read, neither early
nor out of a cache."""
import pytest
import torch

pytestmark = pytest.mark.gpu
bf16, f32 = torch.bfloat16, torch.float32
ROUNDS = 12


@pytest.fixture(scope="module")
def q():
    import transformer_ffn_block_gb300 as q
    return q


def _on_device(seed, *shape, std=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.empty(*shape, device="cuda").normal_(0.0, std, generator=g).to(bf16)


def _chain(q, M, C, sync):
    """x -> norm -> linear -> linear with the output as weights, bias and residual -> gated with it as weights
    -> norm with it as gain and shift -> the norm's backward with it as gain -> the linear's backward: ROUNDS
    times over the same buffers, on other inputs each time.  Returns every round's results."""
    new = lambda *s, t=bf16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    w, ones = _on_device(1, C, C, std=C ** -0.5), torch.ones(C, dtype=bf16, device="cuda")
    y, z, a, yy, dx = (new(M, C) for _ in range(5))
    g = new(M, C // 2)
    mean, rstd, dgain, dshift, db = new(M, t=f32), new(M, t=f32), new(C, t=f32), new(C, t=f32), new(C, t=f32)
    w2, b = new(C, C), new(M, C)
    size = max(q.qffn_linear_workspace_size(M, C, C), q.qffn_linear_workspace_size(C, C, C),
               q.qffn_gated_linear_workspace_size(M, C, C // 2), q.qffn_norm_backward_workspace_size(M, C),
               q.qffn_linear_backward_workspace_size(M, C, C))
    ws = new(size, t=torch.uint8)
    inputs = [(_on_device(10 + i, M, C), _on_device(40 + i, C, C, std=0.05)) for i in range(ROUNDS)]
    out = []

    def step():
        if sync:
            torch.cuda.synchronize()

    torch.cuda.synchronize()
    for x, v in inputs:
        q.qffn_layernorm_absmax(None, y, mean, rstd, None, None, x, ones, None, 1e-5, M, C)
        step()
        q.qffn_linear(a, z, y, w, None, None, q.QFFN_ACT_GELU, M, C, C, ws)
        step()
        q.qffn_linear(w2, None, v, w, None, None, q.QFFN_ACT_NONE, C, C, C, ws)          # the weights of the next call
        step()
        q.qffn_linear(b, None, a, w2, w2[0], a, q.QFFN_ACT_NONE, M, C, C, ws)
        step()
        q.qffn_gated_linear(g, b, w2, q.QFFN_ACT_SILU, M, C, C // 2, ws)
        step()
        q.qffn_linear(yy, None, v[:M] if M <= C else x, w, None, None, q.QFFN_ACT_NONE, M, C, C, ws)
        step()
        q.qffn_layernorm_absmax(None, y, mean, rstd, None, None, b, yy[0], yy[M - 1], 1e-5, M, C)
        step()
        q.qffn_layernorm_backward(dx, dgain, dshift, None, yy, None, b, mean, rstd, y[0], M, C, False, ws)
        step()
        q.qffn_linear_backward(yy, w2, db, dx, z, y, w, q.QFFN_ACT_GELU, M, C, C, False, ws)
        step()
        q.qffn_linear(b, None, yy, w2, None, None, q.QFFN_ACT_NONE, M, C, C, ws)
        step()
        out.append([t.clone() for t in (y, a, b, g, yy, dx, w2, dgain, dshift, db)])
    torch.cuda.synchronize()
    q.qffn_check_status()
    return out


@pytest.mark.parametrize("M,C", [(1, 512), (1, 2048), (16, 1024), (24, 2048), (64, 1024), (200, 512), (300, 1024), (700, 1024)])
def test_each_call_on_the_results_of_the_one_before(q, M, C):
    want = _chain(q, M, C, True)
    for _ in range(3):
        for i, (got, ref) in enumerate(zip(_chain(q, M, C, False), want)):
            for j, (s, t) in enumerate(zip(got, ref)):
                assert torch.equal(s.view(torch.uint8), t.view(torch.uint8)), (i, j)


@pytest.mark.parametrize("M,C", [(40, 512), (300, 1024)])
def test_fp8_calls_on_the_results_of_the_one_before(q, M, C):
    """Quantise the output of a linear layer, use its codes as activations, then as weights, with its first row as bias."""
    new = lambda *s, t=bf16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    w = _on_device(1, C, C, std=C ** -0.5)
    a, b, c = new(C, C), new(M, C), new(M, C)
    aq, bq = new(C, C, t=torch.uint8), new(M, C, t=torch.uint8)
    sa, sb = new(2, t=f32), new(2, t=f32)
    ws = new(max(q.qffn_linear_workspace_size(C, C, C), q.qffn_linear_fp8_workspace_size(M, C, C), 256), t=torch.uint8)
    inputs = [_on_device(10 + i, C, C) for i in range(ROUNDS)]

    def chain(sync):
        out = []
        step = torch.cuda.synchronize if sync else (lambda: None)
        for x in inputs:
            q.qffn_linear(a, None, x, w, None, None, q.QFFN_ACT_SILU, C, C, C, ws)
            step()
            q.qffn_absmax(sa, a, C * C)
            q.qffn_quantize(aq, sa, a, C * C)
            step()
            q.qffn_linear_fp8(b, None, aq, sa[1:], aq, sa[1:], a[0], a, q.QFFN_ACT_RELU, M, C, C, ws)
            step()
            q.qffn_absmax(sb, b, M * C)
            q.qffn_qmm(c, bq, sb, b, a[1], aq, sa[1:], M, C, C)
            step()
            out.append([t.clone() for t in (a, b, c, aq, bq)])
        torch.cuda.synchronize()
        q.qffn_check_status()
        return out

    want = chain(True)
    for _ in range(3):
        for got, ref in zip(chain(False), want):
            for s, t in zip(got, ref):
                assert torch.equal(s.view(torch.uint8), t.view(torch.uint8))


def test_decode_on_weights_written_just_before(q):
    """The decode without the stable-weights flag reads its records behind the kernel that writes them."""
    C, H = 1024, 2816
    new = lambda *s, t=bf16: torch.zeros(*s, dtype=t, device="cuda")  # noqa: E731
    codes = [new(H, C, t=torch.uint8), new(H, C, t=torch.uint8), new(C, H, t=torch.uint8)]
    scales = [new(H, t=f32), new(H, t=f32), new(C, t=f32)]
    out, x = new(C), new(1, C)
    ws = new(q.qffn_decode_workspace_size(C, H), t=torch.uint8)
    lw = _on_device(2, C, C, std=C ** -0.5)
    lws = new(q.qffn_linear_workspace_size(1, C, C), t=torch.uint8)
    sets = [[_on_device(100 + 3 * i + k, *c.shape, std=0.05) for k, c in enumerate(codes)] for i in range(ROUNDS)]
    xs = [_on_device(200 + i, 1, C) for i in range(ROUNDS)]

    def chain(sync):
        res = []
        step = torch.cuda.synchronize if sync else (lambda: None)
        for rows, xi in zip(sets, xs):
            q.qffn_linear(x, None, xi, lw, None, None, q.QFFN_ACT_NONE, 1, C, C, lws)
            for c, s, w in reversed(list(zip(codes, scales, rows))):
                q.qffn_quantize_rows(c, s, w, *w.shape)
                step()
            q.qffn_decode_forward(out, x, codes[0], scales[0], codes[1], scales[1], codes[2], scales[2], C, H, ws)
            step()
            res.append(out.clone())
        torch.cuda.synchronize()
        return res

    want = chain(True)
    for _ in range(3):
        for s, t in zip(chain(False), want):
            assert torch.equal(s.view(torch.int16), t.view(torch.int16))
