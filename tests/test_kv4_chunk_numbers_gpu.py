"""What kv4_attention over chunks of a prompt does with values that are no numbers, wherever in the keys they are. Which
outputs are NaN follows from the mask alone."""
import pytest
import torch

import memory_bound_weight_gb300 as mbw
from test_kv4_chunk_gpu import cache_of, run
from test_kv4_gpu import gen, new_cache, normal

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


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("value", [66000.0, 2e5, -7e4, 9e5])
def test_a_value_beyond_fp16_is_nan_to_the_queries_that_see_it(which, value):
    """Its token's group reads as NaN; to the queries of the same tile before it, it is not there."""
    ctx, nq, hq, hk, d, at, page = 500, 160, 16, 2, 128, 420, 16
    cache, table, _, g = cache_of(91, [ctx], page, hk, d, 64, lambda g, n: (normal(g, n, hk, d), normal(g, n, hk, d)))
    q = normal(g, nq, hq, d)
    without, _ = run(cache, q, table, [ctx], [0, nq])
    k, v = (x.clone() for x in mbw.kv4_gather(cache, slot_of(table, 0, at, page)))
    (k if which == "k" else v)[0, 0, 3] = value
    mbw.kv4_append(cache, k, v, slot_of(table, 0, at, page))
    for window in (0, 30):
        out, _ = run(cache, q, table, [ctx], [0, nq], window=window)
        pos = torch.arange(ctx - nq, ctx, device="cuda")
        see = (pos >= at) & (pos < at + window if window else pos >= 0)
        want = torch.zeros(nq, hq, d, dtype=torch.bool, device="cuda")
        want[see, :hq // 2, :d if which == "k" else 64] = True
        assert torch.equal(out.isnan(), want)
        if not window:
            assert torch.equal(out[~see], without[~see])


@pytest.mark.parametrize("fill", [0x7B, 0xF8, 0x6F, 0xFE, 0x7C, 0x00])
@pytest.mark.parametrize("d,group", [(64, 32), (128, 64)])
def test_bytes_that_were_never_written_do_not_enter(fill, d, group):
    """The tokens before every query's window were never appended: their scales and minima are whatever the bytes are."""
    ctx, nq, hq, hk, first, page, window = 700, 150, 16, 2, 507, 16, 40
    outs = []
    for byte in (fill, 0x31):
        g = gen(92)
        cache = new_cache(-(-ctx // page), page, hk, d, group, fill=byte)
        k, v, q = normal(g, ctx - first, hk, d), normal(g, ctx - first, hk, d), normal(g, nq, hq, d)
        mbw.kv4_append(cache, k, v, torch.arange(first, ctx, device="cuda"))
        table = torch.arange(-(-ctx // page), dtype=torch.int32, device="cuda")[None].contiguous()
        outs.append(run(cache, q, table, [ctx], [0, nq], window=window))
    assert outs[0][0].isfinite().all() and torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
