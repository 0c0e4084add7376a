"""kv4_attention with windows of any size, beside requests with more queries than tokens: a window that holds every position
changes nothing."""
import pytest
import torch

import memory_bound_weight_gb300 as mbw
from test_kv4_gpu import filled, normal

pytestmark = pytest.mark.gpu

MAX_DIM = (1 << 31) - (1 << 16)  # MBW_MAX_DIM


@pytest.mark.parametrize("others", [3, 2500])  # chunks on average; single tokens on average
@pytest.mark.parametrize("d,group", [(64, 32), (256, 64)])
@pytest.mark.parametrize("space", ["full", "none"])
def test_windows_near_the_largest_size(others, d, group, space):
    """A request of 10 tokens and 70000 queries: the first sits 69990 places before the first token."""
    ctx, nq = [10] + [40 + i % 100 for i in range(others)], [70000] + [1 + i % 2 for i in range(others)]
    cache, table, _, g = filled(94, ctx, 16, 1, d, group)
    starts = [0]
    for n in nq:
        starts.append(starts[-1] + n)
    q = normal(g, starts[-1], 1, d)
    c, s = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (ctx, starts))
    ws = mbw.kv4_attention_workspace(d) if space == "full" else None
    want, want_lse = mbw.kv4_attention(cache, q, table, c, s, return_lse=True, workspace=ws)
    assert want[:69990].eq(0).all() and want_lse[:69990].eq(-float("inf")).all() and want_lse[69990:].isfinite().all()
    for window in (1000, MAX_DIM - 65536, MAX_DIM - 1, MAX_DIM, (1 << 31) - 1, 1 << 40):
        out, lse = mbw.kv4_attention(cache, q, table, c, s, window=window, return_lse=True, workspace=ws)
        assert torch.equal(out, want) and torch.equal(lse, want_lse), window
