"""Weight blocks outside the binary16 range in the fused and the experts'
prefill products: reported where an output reads them, and only there."""
import struct

import pytest
import torch

from operator_refs import NONE, SILU, random_weight

pytestmark = pytest.mark.gpu

RANGE = 9


def spoil(dsq, w, qtype, K, row, unit):
    """Gives one block of a packed row a scale whose values pass 65520."""
    w.view(-1)[row * dsq.dsq_row_bytes(qtype, K) + unit * (272 if qtype == 8 else 144):][:2] = torch.tensor(
        list(struct.pack("<e", 2000.0)), dtype=torch.uint8, device="cuda")
    if qtype == 12:   # the largest sub-block scales, so that no code can hide it
        w.view(-1)[row * dsq.dsq_row_bytes(qtype, K) + unit * 144 + 4:][:4] = 63


def weight(dsq, qtype, rows, K, seed, bad=()):
    w = random_weight(qtype, rows, K, seed)
    for row, unit in bad:
        spoil(dsq, w, qtype, K, row, unit)
    return w


@pytest.mark.parametrize("qtype", [8, 12])
# the small kernels, K cut over SMs, whole tiles, a split last wave
@pytest.mark.parametrize("M,N,K", [(1, 100, 512), (6, 100, 512), (40, 100, 1024), (300, 8192, 512), (2048, 5120, 512)])
def test_fused_prefill(dsq, qtype, M, N, K):
    x, y = torch.randn(M, K, device="cuda"), torch.empty(M, N, device="cuda")
    good = weight(dsq, qtype, N, K, 1)
    bad = weight(dsq, qtype, N, K, 1, [(N - 3, K // 256 - 1)])
    for w0, w1, want in ((good, None, 0), (bad, None, RANGE), (good, good, 0), (good, bad, RANGE), (bad, good, RANGE)):
        need = dsq.dsq_prefill_fused_workspace_bytes(qtype, w1 is not None, N, K, M)
        ws = torch.empty(need, dtype=torch.uint8, device="cuda")
        dsq.dsq_gemm_prefill_fused(qtype, w0, w1, N, K, x, M, NONE, None, None, None, y, ws, need)
        assert dsq.dsq_device_status() == want
        assert y[:, :N - 3].isfinite().all() and y[:, N - 2:].isfinite().all()
        assert y[:, N - 3].isfinite().all() == (want == 0)


@pytest.mark.parametrize("qtype", [8, 12])
@pytest.mark.parametrize("gated", [False, True])
@pytest.mark.parametrize("N", [1, 100, 128, 200, 300])
def test_experts_report_their_own_rows_only(dsq, qtype, gated, N):
    E, K, P = 4, 512, 70
    x = torch.randn(P, K, device="cuda")
    offsets = torch.tensor([0, 30, 30, 70, 70], dtype=torch.int32, device="cuda")   # experts 1 and 3 have no rows
    good = weight(dsq, qtype, E * N, K, 2)
    own = [[(0, 0)], [(N - 1, 1)], [(2 * N, 1)], [(3 * N - 1, 0)]]
    others = [[(e * N + r, u) for e in (1, 3) for r in {0, N // 2, N - 1} for u in (0, 1)]]
    want_y = None
    for bad, want in [([], 0)] + [(b, RANGE) for b in own] + [(b, 0) for b in others]:
        for which in range(2 if gated and bad else 1):
            w = [weight(dsq, qtype, E * N, K, 2, bad) if i == which else good for i in range(2)]
            need = dsq.dsq_experts_workspace_bytes(qtype, gated, E, N, K, P)
            ws, y = torch.empty(need, dtype=torch.uint8, device="cuda"), torch.empty(P, N, device="cuda")
            dsq.dsq_gemm_experts(qtype, w[0], w[1] if gated else None, E, N, K, offsets, None, 1, P, x, P, SILU, None, None, y, ws, need)
            assert dsq.dsq_device_status() == want, (bad, which)
            if want == 0:
                want_y = y if want_y is None else want_y
                assert torch.equal(y, want_y)
            else:
                row = bad[0][0]
                assert not y[slice(0, 30) if row < N else slice(30, 70), row % N].isfinite().all()
