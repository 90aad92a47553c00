"""How many bits the sums of the linear and gated layers are kept in: the error of a whole result in the mean
square, which sums held, joined or exchanged in bf16 raise although every element stays within its bound."""
import pytest
import torch

import plain_ops as P

gpu = pytest.mark.gpu
bf16, f32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module")
def q():
    import transformer_ffn_block_gb300 as q
    return q


# An fp32 error before a rounding moves some values across the middle between two bf16 numbers.  Such a value's error
# keeps its size (nearly half a step on either side) and changes sign, so the sum of squares changes only through its
# products with the other errors.  At most 2 * 1.5e-5 / 2^-8 = 0.8 % of the values are that close (the slopes' 4 ACT_REL
# is the largest such error here), and with n independent errors the change is 2 sqrt(0.008 / n) in the mean: 1.1 % for
# the smallest n here (264), under 0.3 % for most.  3 % bounds it; sums exchanged in bf16 add 25 % and more.
FLIPS = 1.03


def _close(got, exact, result, terms):
    size = exact.norm()
    model = ((result.to(bf16).double() - exact).norm() / size).item() ** 2
    return ((got.double() - exact).norm() / size).item() ** 2 <= FLIPS * model + (terms * 2.0 ** -24) ** 2


def within_one_rounding(got, exact, terms):
    """Whether got's error in the mean square is that of rounding `exact` to bf16 once, beside fp32 sums.

    A sum of `terms` products makes as many additions, each off by at most half an fp32 unit (2^-24) of a partial
    sum, which in the mean square is no larger than the whole; that error and the rounding's are independent."""
    return _close(got, exact, exact, terms)


def after_rounded_dz(got, exact, rounded, terms):
    """The same for a product of dz, which the tensor cores take rounded to bf16: `rounded` is the product of the
    rounded dz in 64 bits, so the result is that, rounded once more."""
    return _close(got, exact, rounded, terms)


def _t(seed, *shape, std=1.0, device="cuda"):
    g = torch.Generator(device=device).manual_seed(seed)
    return torch.empty(*shape, device=device).normal_(0.0, std, generator=g).to(bf16)


@pytest.mark.parametrize("K", [2048, 8272, 14336])
def test_the_rule_tells_bf16_sums_from_fp32_sums(K):
    x, w = _t(1, 24, K, device="cpu"), _t(2, 200, K, std=K ** -0.5, device="cpu")
    exact = x.double() @ w.double().t()
    parts = [(a.float() @ b.float().t()) for a, b in zip(x.chunk(2, 1), w.chunk(2, 1))]
    assert within_one_rounding((parts[0] + parts[1]).to(bf16), exact, K)
    assert not within_one_rounding((parts[0].to(bf16).float() + parts[1]).to(bf16), exact, K)   # one part exchanged in bf16
    assert not within_one_rounding((parts[0].to(bf16) + parts[1].to(bf16)), exact, K)           # a join of bf16 parts
    dz = _t(3, 200, 24, std=1e-3, device="cpu").double() * 0.7317
    ex, ro = dz @ x.double(), dz.to(bf16).double() @ x.double()
    assert after_rounded_dz(ro.to(bf16), ex, ro, 24)
    half = [a.t() @ b.double() for a, b in zip(dz.to(bf16).double().t().chunk(2, 0), x.chunk(2, 0))]
    assert not after_rounded_dz((half[0].to(bf16).double() + half[1]).to(bf16), ex, ro, 24)


# every form: streamed weights, few rows over 1 to 8 parts of K, whole and narrow units, parts of K joined, exchanged
FORWARD = [(1, 264, 8272), (16, 1000, 4104), (20, 4624, 8336), (33, 1072, 4392), (64, 4096, 14336), (40, 512, 8192), (104, 792, 2632),
           (165, 584, 2192), (300, 264, 8200), (487, 168, 2960), (512, 2048, 8192), (333, 4096, 2048), (1316, 520, 7032),
           (2304, 2568, 2048)]


@gpu
@pytest.mark.parametrize("M,N,K", FORWARD)
@pytest.mark.parametrize("fp8", [False, True])
def test_linear_sums(q, M, N, K, fp8):
    K = (K + 15) // 16 * 16 if fp8 else K
    x, w, b, res = _t(1, M, K), _t(2, N, K, std=K ** -0.5), _t(3, N), _t(4, M, N)
    out, z = torch.empty(M, N, dtype=bf16, device="cuda"), torch.empty(M, N, dtype=bf16, device="cuda")
    if fp8:
        x, w, s = x.to(torch.float8_e4m3fn), (w * 64).to(torch.float8_e4m3fn), torch.tensor([0.5, 1 / 32], device="cuda")
        ws = torch.empty(q.qffn_linear_fp8_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")
        q.qffn_linear_fp8(out, z, x, s[0:1], w, s[1:2], b, res, q.QFFN_ACT_SILU, M, N, K, ws)
    else:
        ws = torch.empty(q.qffn_linear_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")
        q.qffn_linear(out, z, x, w, b, res, q.QFFN_ACT_SILU, M, N, K, ws)
    q.qffn_check_status()
    zz = (x.double() @ w.double().t()) * (1 / 64 if fp8 else 1.0) + b.double()
    assert within_one_rounding(z, zz, K)
    assert within_one_rounding(out, P.act(zz, "silu") + res.double(), K)


@gpu
@pytest.mark.parametrize("M,C,H", [(1, 8272, 264), (16, 2048, 520), (24, 7600, 2312), (64, 4096, 1408), (99, 2600, 392), (300, 8192, 264),
                                   (512, 4096, 1024), (2304, 2048, 1280)])
def test_gated_sums(q, M, C, H):
    x, w1 = _t(1, M, C), _t(2, 2 * H, C, std=C ** -0.5)
    h = torch.empty(M, H, dtype=bf16, device="cuda")
    ws = torch.empty(q.qffn_gated_linear_workspace_size(M, C, H), dtype=torch.uint8, device="cuda")
    q.qffn_gated_linear(h, x, w1, q.QFFN_ACT_SILU, M, C, H, ws)
    q.qffn_check_status()
    g, u = (x.double() @ v.double().t() for v in w1.chunk(2, 0))
    assert within_one_rounding(h, P.act(g, "silu") * u, 2 * C)


# input gradient of few rows, whole, narrow and over parts; weight gradient from few and from many rows, over parts
BACKWARD = [(2, 4008, 4624), (16, 4096, 1024), (64, 4104, 520), (135, 1432, 3112), (300, 776, 1288), (524, 264, 6664), (3240, 136, 3384),
            (2336, 520, 264), (1111, 4104, 2056), (8200, 136, 264)]


@gpu
@pytest.mark.parametrize("M,N,K", BACKWARD)
@pytest.mark.parametrize("name,accumulate", [("none", False), ("gelu", True), ("silu", False)])
def test_linear_backward_sums(q, M, N, K, name, accumulate):
    dout, z, x, w, old = _t(1, M, N, std=1e-2), _t(2, M, N, std=1.2), _t(3, M, K), _t(4, N, K, std=N ** -0.5), _t(5, N, K, std=1e-2)
    dx, dw, db = torch.empty(M, K, dtype=bf16, device="cuda"), old.clone(), torch.zeros(N, device="cuda")
    ws = torch.empty(q.qffn_linear_backward_workspace_size(M, N, K), dtype=torch.uint8, device="cuda")
    q.qffn_linear_backward(dx, dw, db, dout, z, x, w, getattr(q, "QFFN_ACT_" + name.upper()), M, N, K, accumulate, ws)
    q.qffn_check_status()
    dz = dout.double() if name == "none" else dout.double() * P.act_grad(z.double(), name)
    dzq, add = dz.to(bf16).double(), old.double() if accumulate else 0.0
    assert after_rounded_dz(dx, dz @ w.double(), dzq @ w.double(), N)
    assert after_rounded_dz(dw, dz.t() @ x.double() + add, dzq.t() @ x.double() + add, M)
    # the bias gradient is summed in fp32 from dz before its rounding
    assert ((db.double() - dz.sum(0)).norm() / dz.sum(0).norm()).item() <= (M + 80) * 2.0 ** -24 + 8 * P.ACT_REL


@gpu
@pytest.mark.parametrize("M,C,H", [(2, 4008, 2344), (64, 1024, 2048), (139, 3312, 1248), (533, 3744, 264), (700, 2056, 2504),
                                   (4100, 264, 520)])
@pytest.mark.parametrize("accumulate", [False, True])
def test_gated_backward_sums(q, M, C, H, accumulate):
    dh, x, w1, old = _t(1, M, H, std=1e-2), _t(2, M, C), _t(3, 2 * H, C, std=C ** -0.5), _t(4, 2 * H, C, std=1e-2)
    dx, dw = torch.empty(M, C, dtype=bf16, device="cuda"), old.clone()
    ws = torch.empty(q.qffn_gated_linear_backward_workspace_size(M, C, H), dtype=torch.uint8, device="cuda")
    q.qffn_gated_linear_backward(dx, dw, dh, x, w1, q.QFFN_ACT_SILU, M, C, H, accumulate, ws)
    q.qffn_check_status()
    g, u = (x.double() @ v.double().t() for v in w1.chunk(2, 0))
    dz = torch.cat([dh.double() * u * P.act_grad(g, "silu"), dh.double() * P.act(g, "silu")], 1)
    dzq, add = dz.to(bf16).double(), old.double() if accumulate else 0.0
    assert within_one_rounding(ws[:M * 2 * H * 2].view(bf16).view(M, 2 * H), dz, 2 * C)
    assert after_rounded_dz(dx, dz @ w1.double(), dzq @ w1.double(), 2 * H + C)
    assert after_rounded_dz(dw, dz.t() @ x.double() + add, dzq.t() @ x.double() + add, M + C)
