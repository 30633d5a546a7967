"""The activations of the fused products over their whole range, tails and
special values included, through every kernel that applies them.  The weights
and activations are zeros, so the value an activation meets is the bias."""
import math

import pytest
import torch

from operator_refs import GELU, GELU_TANH, NONE, RELU, SILU, U, quantize

pytestmark = pytest.mark.gpu

K = 512
INF, NAN = float("inf"), float("nan")
SPECIAL = [0.0, -0.0, 1e-45, -1e-45, 1e-30, -1e-30, 1.0, -1.0, 87.2, -87.2, 87.5, -87.5, 88.8, -88.8, 103.9, -103.9, 200.0, -200.0,
           1e13, -1e13, 1.8e19, -1.8e19, 3.4e38, -3.4e38, INF, -INF, NAN]


def values():
    """2500 values: dense about 0 and through the tails, every scale, and the special ones."""
    fine = torch.cat([torch.linspace(-15, 15, 1501), torch.linspace(-110, 110, 500),
                      torch.logspace(-8, 2, 236) * torch.tensor([1.0, -1.0]).repeat(118), -torch.logspace(-8, 2, 236)])
    return torch.cat([fine, torch.tensor(SPECIAL)]).float().cuda()


def exact(v, act):
    v = v.double()
    if act == SILU:
        return v / (1 + torch.exp(-v))
    if act == GELU:
        return 0.5 * v * torch.erfc(-v * math.sqrt(0.5))
    if act == GELU_TANH:   # (1 + tanh u) / 2 = 1 / (1 + exp(-2u)), which does not cancel
        return v / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)))
    return v.clamp(min=0) if act == RELU else v


def bound(v, act):
    """Relative error of the fp32 activation, in units of U.  CUDA documents
    expf within 2 steps (4 U of the value) and the approximate reciprocal within 1 (2 U).
    1 / (1 + exp(-w)) is n (1 / (1 + e)), e = exp(-|w|): e's error passes with a factor of
    at most 1 in all (n = e: 1 / (1 + e); n = 1: e / (1 + e)), the sum adds 1, the
    reciprocal 2, the products with n and v 1 each: 9.
    GELU's tanh form multiplies 2u = v (c1 + c3 v^2), of relative error 4 (a constant,
    the square, the multiply-add, the product), by a slope of at most |2u|.
    GELU: v Phi(v), Phi(-x) = exp(-x^2/2) t Q(t).  The fit 3; t = 1 / (1 + 0.3 x) 3, passed
    with a factor of at most 2.7, so 9 (the logarithmic slope of t Q(t), largest at x = 0); Q's 7
    multiply-adds and rounded coefficients 8 of sum |c_i| t^i <= 1.84 Q: 15; expf 4, the
    rounded square x^2 / 2 U in the exponent; three products: 34 + x^2 / 2.  Where 1 less
    that is taken, it is at most half, so the error is no larger, and one more; 37 in all."""
    x = v.double().abs()
    if act == SILU:
        return torch.full_like(x, 9)
    if act == GELU:
        return 37 + x * x / 2
    if act == GELU_TANH:
        return 9 + 4 * 2 * math.sqrt(2 / math.pi) * (x + 0.044715 * x ** 3)
    return torch.zeros_like(x)   # exact, at infinity too


def check(y, v, act):
    """y: rows of activations of v."""
    want = exact(v, act)
    some = want.isfinite()
    # the limit at +-infinity and NaN as the formula gives them
    assert torch.equal(y[:, ~some].isnan(), want[~some].isnan().expand_as(y[:, ~some])), act
    assert torch.equal(y[:, v == INF], torch.full_like(y[:, v == INF], INF))
    assert act not in (NONE, RELU) or (y[:, v == -INF] == (0 if act == RELU else -INF)).all()
    b = bound(v, act).clamp(max=2.0 ** 22)   # far tails of the tanh form: below 2^-126 below
    # a factor on v below 2^-126 has fewer bits in fp32 and may come out as 0
    floor = v.double().abs().clamp(min=1, max=256) * 2.0 ** -125
    tol = 1.01 * b * U * want.abs() + torch.where(want.abs() < floor, floor, 0.0)
    err = (y.double() - want).abs()
    bad = ~(err <= tol) & some
    assert not bad.any(), (act, v[bad.any(0)][:5].tolist(), y[bad][:5].tolist(), want[bad.any(0)][:5].tolist())


def zero_weight(dsq, qtype, rows):
    return torch.zeros(rows * dsq.dsq_row_bytes(qtype, K), dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("act", [NONE, SILU, GELU, GELU_TANH, RELU])
@pytest.mark.parametrize("qtype", [8, 12])
# one token by rows and by boxes, two tokens, the tensor cores
@pytest.mark.parametrize("N,M", [(1000, 1), (2500, 1), (2500, 2), (2500, 8), (6000, 1)])
def test_decode(dsq, qtype, act, N, M):
    v = values().repeat(3)[:N].contiguous()
    w = zero_weight(dsq, qtype, N)
    q = quantize(dsq, torch.zeros(M, K, device="cuda"))
    y = torch.empty(M, N, device="cuda")
    dsq.dsq_gemv_fused(qtype, w, None, N, K, M, *q, act, v, None, None, y)
    check(y, v, act)
    ones = torch.ones(N, device="cuda")
    dsq.dsq_gemv_fused(qtype, w, w, N, K, M, *q, act, v, ones, None, y)
    check(y, v, act)
    assert dsq.dsq_device_status() == 0


@pytest.mark.parametrize("act", [NONE, SILU, GELU, GELU_TANH, RELU])
@pytest.mark.parametrize("qtype", [8, 12])
# the small kernels, K cut over SMs, whole tiles
@pytest.mark.parametrize("M,rep", [(1, 1), (5, 1), (40, 1), (300, 8)])
def test_prefill(dsq, qtype, act, M, rep):
    v = values().repeat(rep).contiguous()
    N = v.numel()
    w = zero_weight(dsq, qtype, N)
    x, ones, y = torch.zeros(M, K, device="cuda"), torch.ones(N, device="cuda"), torch.empty(M, N, device="cuda")
    for w1, b1 in ((None, None), (w, ones)):
        need = dsq.dsq_prefill_fused_workspace_bytes(qtype, w1 is not None, N, K, M)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        dsq.dsq_gemm_prefill_fused(qtype, w, w1, N, K, x, M, act, v, b1, None, y, ws, need)
        check(y, v, act)
    assert dsq.dsq_device_status() == 0


@pytest.mark.parametrize("act", [NONE, SILU, GELU, GELU_TANH, RELU])
@pytest.mark.parametrize("qtype", [8, 12])
@pytest.mark.parametrize("P", [2, 40])
def test_experts(dsq, qtype, act, P):
    v, E = values(), 2
    N = v.numel()
    w = zero_weight(dsq, qtype, E * N)
    offsets = torch.tensor([0, P // 2, P], dtype=torch.int32, device="cuda")
    x, y = torch.zeros(P, K, device="cuda"), torch.empty(P, N, device="cuda")
    bias = v.repeat(E)
    dsq.dsq_gemv_experts(qtype, w, None, E, N, K, offsets, None, 1, P, *quantize(dsq, x), P, act, bias, None, y)
    check(y, v, act)
    need = dsq.dsq_experts_workspace_bytes(qtype, False, E, N, K, P)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
    y.zero_()
    dsq.dsq_gemm_experts(qtype, w, None, E, N, K, offsets, None, 1, P, x, P, act, bias, None, y, ws, need)
    check(y, v, act)
    assert dsq.dsq_device_status() == 0
