"""kv4_attention_shared in a chain of calls that write, right in front of it and to the same places each time, all that it reads:
queries, lengths, the block table and pages. Its second kernel starts before the first has ended, and must read what is new."""
import pytest
import torch

import memory_bound_weight_gb300 as mbw
from test_kv4_gpu import gen, new_cache, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,T,d", [(64, 1, 128), (40, 3, 64), (6, 8, 128)])
def test_all_that_is_read_changes_in_front_of_every_call(B, T, d):
    hq, hk, page, group, prefix = 32, 8, 16, 32, 9600
    common, own = prefix // page, 6
    g = gen(B + T)
    total = common + B * own
    cache = new_cache(total, page, hk, d, group)
    for at in range(0, total * page, 4096):
        n = min(4096, total * page - at)
        mbw.kv4_append(cache, normal(g, n, hk, d), normal(g, n, hk, d), torch.arange(at, at + n, device="cuda"))
    front = torch.arange(common, dtype=torch.int32, device="cuda").repeat(B, 1)
    rounds = []
    for i in range(5):
        mine = common + torch.randperm(B * own, generator=g, device="cuda").to(torch.int32).view(B, own)
        ctx = (prefix + torch.randint(T, own * page, (B,), generator=g, device="cuda")).to(torch.int32)
        last = mine.gather(1, ((ctx - 1 - prefix) // page).long()[:, None])[:, 0].long() * page + (ctx.long() - 1) % page
        rounds.append((normal(g, B * T, hq, d), torch.cat((front, mine), 1).contiguous(), ctx, last,
                       normal(g, B, hk, d) * 3, normal(g, B, hk, d) * 3))
    q, table, ctx, slots, k, v = (torch.empty_like(x) for x in rounds[0])
    starts = None if T == 1 else torch.arange(0, B * T + 1, T, dtype=torch.int32, device="cuda")
    ws = mbw.kv4_attention_shared_workspace(d, B * T, hq)

    def step(r, wait=False):
        for to, x in zip((q, table, ctx, slots, k, v), r):
            to.copy_(x)
        mbw.kv4_append(cache, k, v, slots)
        if wait:
            torch.cuda.synchronize()
        n = mbw.launch_count()
        got = mbw.kv4_attention_shared(cache, q, table, ctx, prefix, starts, return_lse=True, workspace=ws)
        assert mbw.launch_count() == n + 2
        return got

    pages = cache.pages.clone()
    want = [step(r, wait=True) for r in rounds]
    torch.cuda.synchronize()
    cache.pages.copy_(pages)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            captured = [step(r) for r in rounds]
    for _ in range(6):
        cache.pages.copy_(pages)
        got = [step(r) for r in rounds]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
        cache.pages.copy_(pages)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(captured, want):
            assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
