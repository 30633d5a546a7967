"""Kernels one behind the other: each reads what the one before has just
written, in buffers that held other values a moment ago.  A chain captured into
a graph and replayed on changing inputs gives what the same calls give with the
device waited for after each."""
import pytest
import torch

from operator_refs import GELU, NONE, SILU, random_weight

pytestmark = pytest.mark.gpu

K, N = 2048, 1024


class State:
    def __init__(self, dsq, qtype, M):
        e = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype, device="cuda")  # noqa: E731
        codes = lambda n: (e(M, n, dtype=torch.int8), e(M, n // 32), e(M, n // 32, dtype=torch.int32))  # noqa: E731
        self.dsq, self.qtype, self.M = dsq, qtype, M
        self.h, self.b = e(M, K), e(M, K)
        self.w_pre = torch.rand(K, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda") + 0.5
        self.up, self.gate, self.down = (random_weight(qtype, n, k, s) for n, k, s in ((N, K, 2), (N, K, 3), (K, N, 4)))
        self.h1, self.x, self.mid, self.mid2, self.out = e(M, K), e(M, K), e(M, N), e(M, N), e(M, K)
        self.q, self.mq = codes(K), codes(N)
        need = max(dsq.dsq_prefill_fused_workspace_bytes(qtype, True, N, K, M), dsq.dsq_prefill_workspace_bytes(qtype, N, K, M),
                   dsq.dsq_prefill_workspace_bytes(qtype, K, N, M), dsq.dsq_prefill_grouped_workspace_bytes(qtype, [N, N], K, M))
        self.ws, self.need = e(need, dtype=torch.uint8), need

    def norm(self, codes):
        self.dsq.dsq_norm_block(self.h, self.b, None, 0, None, 1.0, self.w_pre, 1e-6, self.M, K, self.h1, None if codes else self.x,
                                *(self.q if codes else (None, None, None)))

    # ------------------------------------------------------------- chains
    def fused_prompt(self):
        d, q, M = self.dsq, self.qtype, self.M
        return [lambda: self.norm(False),
                lambda: d.dsq_gemm_prefill_fused(q, self.gate, self.up, N, K, self.x, M, SILU, None, None, None, self.mid, self.ws, self.need),
                lambda: d.dsq_gemm_prefill_fused(q, self.down, None, K, N, self.mid, M, GELU, None, None, self.h1, self.out, self.ws, self.need)]

    def plain_prompt(self):
        d, q, M = self.dsq, self.qtype, self.M
        return [lambda: self.norm(False),
                lambda: d.dsq_gemm_prefill_grouped(q, [self.gate, self.up], [N, N], K, self.x, M, [self.mid, self.mid2], self.ws, self.need),
                lambda: d.dsq_gemm_prefill(q, self.down, K, N, self.mid, M, self.out, self.ws, self.need)]

    def fused_decode(self):
        d, q, M = self.dsq, self.qtype, self.M
        return [lambda: self.norm(True),
                lambda: d.dsq_gemv_fused(q, self.gate, self.up, N, K, M, *self.q, SILU, None, None, None, self.mid),
                lambda: d.dsq_quantize_act_q8(self.mid, M, N, *self.mq),
                lambda: d.dsq_gemv_fused(q, self.down, None, K, N, M, *self.mq, NONE, None, None, self.h1, self.out)]

    def plain_decode(self):
        d, q, M = self.dsq, self.qtype, self.M
        return [lambda: self.norm(True),
                lambda: d.dsq_gemv_tokens(q, self.gate, N, self.up, N, K, M, *self.q, self.mid, self.mid2),
                lambda: d.dsq_quantize_act_q8(self.mid, M, N, *self.mq),
                lambda: d.dsq_gemv_tokens(q, self.down, K, None, 0, N, M, *self.mq, self.out, None)]

    def one_token(self):
        d, q = self.dsq, self.qtype
        return [lambda: self.norm(False),
                lambda: d.dsq_quantize_act_q8(self.x, 1, K, *self.q),
                lambda: d.dsq_gemv_paired(q, self.gate, N, self.up, N, K, *self.q, self.mid, self.mid2),
                lambda: d.dsq_gemv_f32(q, self.down, K, N, self.mid, self.out)]


CHAINS = [("one_token", 1)] + [(c, M) for c in ("fused_decode", "plain_decode") for M in (1, 3, 8)] + \
         [(c, M) for c in ("fused_prompt", "plain_prompt") for M in (1, 5, 40, 300)]


@pytest.mark.parametrize("qtype", [8, 12])
@pytest.mark.parametrize("chain,M", CHAINS)
def test_chain_in_a_graph_on_changing_inputs(dsq, qtype, chain, M):
    s = State(dsq, qtype, M)
    calls = getattr(s, chain)()
    g = torch.Generator(device="cuda").manual_seed(M)
    inputs = [(torch.randn(M, K, generator=g, device="cuda"), torch.randn(M, K, generator=g, device="cuda")) for _ in range(6)]
    want = []
    for h, b in inputs:
        s.h.copy_(h)
        s.b.copy_(b)
        for call in calls:
            call()
            torch.cuda.synchronize()
        want.append(s.out.clone())
    assert not any(torch.equal(want[0], w) for w in want[1:])
    stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        for call in calls:
            call()
    got = []
    with torch.cuda.stream(stream):
        for h, b in inputs * 3:
            s.h.copy_(h)
            s.b.copy_(b)
            graph.replay()
            got.append(s.out.clone())
    torch.cuda.synchronize()
    for i, y in enumerate(got):
        assert torch.equal(y, want[i % len(want)]), i
    assert dsq.dsq_device_status() == 0
