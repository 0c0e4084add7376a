"""kv4_attention with query offsets that fall or leave the queries: reported, nothing but the outputs written, and the
workspace ready for the next call."""
import pytest
import torch

import memory_bound_weight_gb300 as mbw
from test_kv4_gpu import gen, new_cache, normal

pytestmark = pytest.mark.gpu

GUARD = 1 << 20


def guarded_workspace(d):
    """A workspace of the needed size and not a byte more, and bytes behind it that show a write."""
    n = mbw.kv4_attention_workspace(d).numel()
    whole = torch.zeros(n + 8 * GUARD, dtype=torch.uint8, device="cuda")
    whole[n:] = 0xA5
    return whole[:n], whole[n:]


# requests, queries, query heads, KV heads, head dimension, tokens of the last request. Where q_starts is 0, T, 0, T, ...
# every other request has all the queries: many more (request, head, tile) items than a call of T queries has room for.
CASES = [
    (2001, 76, 1, 1, 128, 200704),   # few items, cut over CTAs; the last one long
    (4001, 40, 2, 2, 64, 100000),
    (301, 700, 8, 4, 128, 30000),    # many items, a warp each
    (21, 900, 16, 4, 64, 5000),      # chunks, up to 32 requests
    (61, 3000, 16, 4, 128, 5000),    # chunks, more requests
]


@pytest.mark.parametrize("B,T,hq,hk,d,last", CASES)
@pytest.mark.parametrize("kind", ["fall", "one fall", "outside"])
def test_offsets_that_fall_or_leave_the_queries(B, T, hq, hk, d, last, kind):
    page, g = 1024, gen(93)
    cache = new_cache(2, page, hk, d, 64)
    mbw.kv4_append(cache, normal(g, 2 * page, hk, d), normal(g, 2 * page, hk, d), torch.arange(2 * page, device="cuda"))
    ctx = torch.full((B,), 16, dtype=torch.int32)
    ctx[-1] = last
    table = torch.zeros(B, -(-last // page), dtype=torch.int32, device="cuda")  # every page is page 0
    good = torch.arange(B + 1, dtype=torch.int64) * T // B
    starts = good.clone()
    if kind == "fall":
        starts[0::2], starts[1::2] = 0, T
    elif kind == "one fall":
        starts[B // 2] = T
    else:
        starts[0], starts[-1] = -7, T + 1000
    q = normal(g, T, hq, d)
    ws, guard = guarded_workspace(d)
    ctx, good, starts = ctx.cuda(), good.int().cuda(), starts.int().cuda()
    want, want_lse = mbw.kv4_attention(cache, q, table, ctx, good, return_lse=True, workspace=ws)
    mbw.check_device_error()
    for w in (ws, None):
        mbw.kv4_attention(cache, q, table, ctx, starts, workspace=w)
        with pytest.raises(mbw.MbwError) as e:
            mbw.check_device_error()
        assert e.value.status == 8
    assert (guard == 0xA5).all() and not ws[:16384].any()
    out, lse = mbw.kv4_attention(cache, q, table, ctx, good, return_lse=True, workspace=ws)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
