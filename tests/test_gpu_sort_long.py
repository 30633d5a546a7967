"""dsq_moe_sort beyond one cluster's choices: chunks of 2048, longer ones, and
chunks that end inside a warp's turn."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,k,E", [(2731, 6, 64), (8192, 4, 256), (16389, 1, 1024), (262144, 1, 3), (262145, 1, 64), (33001, 8, 1),
                                   (100003, 8, 256), (150001, 6, 1000)])
def test_long_sorts(dsq, T, k, E):
    g = torch.Generator(device="cuda").manual_seed(T)
    n = T * k
    expert = torch.randint(-1, E + 1, (T, k), generator=g, device="cuda", dtype=torch.int32)
    expert[:T // 8] = E // 2   # long runs of one expert
    key = torch.where((expert >= 0) & (expert < E), expert, E).view(-1)
    order = torch.sort(key, stable=True).indices
    count = torch.bincount(key, minlength=E + 1)[:E]
    kept = int(count.sum())
    need = dsq.dsq_moe_sort_workspace_bytes(T, k, E)
    ws = torch.full((need + 256,), 255, dtype=torch.uint8, device="cuda")
    offsets, rows, pos = (torch.full((m + 8,), -7, dtype=torch.int32, device="cuda") for m in (E + 1, n, n))
    for _ in range(2):
        dsq.dsq_moe_sort(expert, T, k, E, offsets, rows, pos, ws, need)
    assert int(offsets[0]) == 0 and torch.equal(offsets[1:E + 1].long(), count.cumsum(0))
    assert torch.equal(rows[:kept].long(), order[:kept]) and (rows[kept:n] == -1).all()
    want = torch.full((n,), -1, device="cuda")
    want[order[:kept]] = torch.arange(kept, device="cuda")
    assert torch.equal(pos[:n].long(), want)
    assert (offsets[E + 1:] == -7).all() and (rows[n:] == -7).all() and (pos[n:] == -7).all() and (ws[need:] == 255).all()
