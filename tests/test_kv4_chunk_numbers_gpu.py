"""What kv4_attention over chunks of a prompt does with values that are no numbers, wherever in the keys they are. Which
outputs are NaN follows from the mask alone."""
import pytest
import torch

import memory_bound_weight_gb300 as mbw
from test_kv4_chunk_gpu import cache_of, run
from test_kv4_gpu import normal

pytestmark = pytest.mark.gpu


def slot_of(table, b, t, page):
    return (table[b, t // page].long() * page + t % page).reshape(1)


@pytest.mark.parametrize("space", ["full", "none"])
@pytest.mark.parametrize("ctx,nq,d,group", [(1152, 128, 64, 32), (900, 200, 128, 64)])
def test_a_nan_value_in_any_tile_of_keys_is_seen(ctx, nq, d, group, space):
    """128 keys a tile, even and odd ones: in each a value that is no number, in its first and its last key."""
    hq, hk, page = 16, 2, 16
    cache, table, _, g = cache_of(90, [ctx], page, hk, d, group, lambda g, n: (normal(g, n, hk, d), normal(g, n, hk, d)))
    q = normal(g, nq, hq, d)
    ws = mbw.kv4_attention_workspace(d) if space == "full" else None
    k, v = normal(g, 1, hk, d), normal(g, 1, hk, d)
    bad = v.clone()
    bad[0, 1, d - 1] = float("nan")  # the last group of the second KV head
    pos = torch.arange(ctx - nq, ctx, device="cuda")
    for at in [t for i in range(0, ctx, 128) for t in (i, min(i + 127, ctx - 1))]:
        mbw.kv4_append(cache, k, bad, slot_of(table, 0, at, page))
        want = torch.zeros(nq, hq, d, dtype=torch.bool, device="cuda")
        want[pos >= at, hq // 2:, d - group:] = True
        for _ in range(5):
            out, lse = run(cache, q, table, [ctx], [0, nq], workspace=ws)
            assert torch.equal(out.isnan(), want), at
            assert lse.isfinite().all()
        mbw.kv4_append(cache, k, v, slot_of(table, 0, at, page))
    assert run(cache, q, table, [ctx], [0, nq], workspace=ws)[0].isfinite().all()
