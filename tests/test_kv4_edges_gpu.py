"""kv4_attention and kv4_append at sizes and arguments where their work is laid out another way: many requests, scales of
zero and below, queries of any size, more tokens than one wave. Tolerances as in test_kv4_gpu.py."""
import pytest
import torch

import kv4_ref as ref
import memory_bound_weight_gb300 as mbw
from test_kv4_gpu import check, filled, gen, new_cache, normal, ulp_bf16

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("hq,hk,d,group", [(8, 2, 128, 64), (4, 2, 64, 32), (6, 1, 256, 64)])
@pytest.mark.parametrize("scale", [0.0, -0.125, 0.3])
def test_single_queries_scales(hq, hk, d, group, scale):
    ctx = [33, 1, 700, 16]
    cache, table, kv, g = filled(70, ctx, 16, hk, d, group)
    q = normal(g, len(ctx), hq, d)
    want = ref.attention(q, kv, ctx, list(range(len(ctx) + 1)), scale)
    c = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    for ws in (None, mbw.kv4_attention_workspace(d)):
        out, lse = mbw.kv4_attention(cache, q, table, c, scale=scale, return_lse=True, workspace=ws)
        check(out, lse, want[0], want[1], want[2])


@pytest.mark.parametrize("size", [2.0 ** -60, 2.0 ** -20, 2.0 ** 20, 2.0 ** 60])
@pytest.mark.parametrize("nq", [1, 3])
def test_queries_of_any_size(size, nq):
    """A power of two moved from the scale to the queries moves nothing in the scores."""
    ctx, hq, hk, d = [90, 300], 8, 2, 128
    cache, table, kv, g = filled(71, ctx, 16, hk, d, 64)
    q = (normal(g, 2 * nq, hq, d).double() * size).bfloat16()
    want = ref.attention(q, kv, ctx, [0, nq, 2 * nq], 0.09 / size)
    out, lse = mbw.kv4_attention(cache, q, table, torch.tensor(ctx, dtype=torch.int32, device="cuda"), scale=0.09 / size,
                                 return_lse=True, workspace=mbw.kv4_attention_workspace(d))
    check(out, lse, want[0], want[1], want[2])


@pytest.mark.parametrize("B", [513, 1100, 2500])
@pytest.mark.parametrize("window", [0, 7])
def test_more_requests_than_threads(B, window):
    """Some requests without a query, some without a token."""
    hq, hk, d = 4, 2, 64
    ctx = [(7 * i * i + 3 * i) % 41 for i in range(B)]
    nq = [0 if i % 5 == 3 else 2 if i % 7 == 2 else 1 for i in range(B)]
    cache, table, kv, g = filled(72, ctx, 16, hk, d, 32)
    starts = [0]
    for n in nq:
        starts.append(starts[-1] + n)
    q = normal(g, starts[-1], hq, d)
    want = ref.attention(q, kv, ctx, starts, d ** -0.5, window)
    c, s = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (ctx, starts))
    for ws in (None, mbw.kv4_attention_workspace(d)):
        out, lse = mbw.kv4_attention(cache, q, table, c, s, window=window, return_lse=True, workspace=ws)
        check(out, lse, want[0], want[1], want[2])


@pytest.mark.parametrize("hq,hk,d,group,rotary,inter", [(7, 1, 128, 64, 128, False), (2, 2, 64, 32, 32, True), (4, 2, 256, 32, 256, False)])
def test_append_of_more_tokens_than_a_wave_with_padding(hq, hk, d, group, rotary, inter):
    T, page = 2600, 16
    g = gen(74)
    cache = new_cache(T // page + 40, page, hk, d, group)
    slots = torch.randperm((T // page + 40) * page, generator=g, device="cuda")[:T].long()
    slots[::17] = -1  # padding tokens are stored nowhere
    pos = torch.randint(0, 500, (T,), generator=g, device="cuda").int()
    cs = mbw.rope_table(500, rotary, device="cuda")
    q, k, v = normal(g, T, hq, d), normal(g, T, hk, d), normal(g, T, hk, d)
    out = mbw.kv4_append(cache, k, v, slots, q=q, positions=pos, cos_sin=cs, interleaved=inter)
    want = ref.rotate(q, cs, pos, inter)
    assert ((ref.f64(out) - want).abs() <= ulp_bf16(want) * (1 + 2.0 ** -10)).all()
    kk = ref.rotate(k, cs, pos, inter).float().bfloat16()
    gk, gv = mbw.kv4_gather(cache, slots)
    for got, x in ((gk, kk), (gv, v)):
        n, s, m = ref.quantize(x, group)
        want = n * s + m
        want[::17] = 0
        assert ((ref.f64(got) - want).abs() <= ulp_bf16(want) * (1 + 2.0 ** -10)).all()


@pytest.mark.parametrize("hk,d", [(5, 128), (8, 64), (3, 256), (1, 256)])
def test_gather_of_many_tokens_is_that_of_few(hk, d):
    """Many tokens take several heads a thread; the values are the same bits."""
    T, page = 12000, 32
    g = gen(75)
    cache = new_cache(T // page + 3, page, hk, d, 32)
    slots = torch.randperm((T // page + 3) * page, generator=g, device="cuda")[:T].long()
    mbw.kv4_append(cache, normal(g, T, hk, d), normal(g, T, hk, d), slots)
    slots[5::31] = -1
    k, v = mbw.kv4_gather(cache, slots)
    assert not torch.isnan(k).any() and (k[5::31] == 0).all() and (v[5::31] == 0).all()
    for i in range(0, T, 700):
        kk, vv = mbw.kv4_gather(cache, slots[i:i + 700].contiguous())
        assert torch.equal(k[i:i + 700], kk) and torch.equal(v[i:i + 700], vv)
