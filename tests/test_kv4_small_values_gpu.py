"""kv4_attention over values of any size, where one key (as the first of a sequence often does) has a weight of its own and
the rest of the result is a sum of many small ones. The bounds are relative to the values: half a step of fp16, 2^-11, of
what a weight multiplies, and as much again for the scores; bf16's half step of the result where it is stored so."""
import pytest
import torch

import kv4_ref as ref
import memory_bound_weight_gb300 as mbw
from test_kv4_gpu import gen, new_cache, normal

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("size", [2.0 ** 13, 1.0, 2.0 ** -7, 2.0 ** -10, 2.0 ** -13, 2.0 ** -16])
@pytest.mark.parametrize("B,nq,ctx,hq,hk,d,group", [
    (64, 1, 2048, 16, 8, 128, 64),   # many items, a warp each
    (48, 3, 1500, 8, 4, 64, 32),
    (1, 1, 6000, 4, 2, 128, 64),     # few, cut over CTAs
    (1, 2, 3000, 2, 1, 256, 32),
    (40, 30, 900, 8, 2, 256, 64),    # tiles of 16 rows
    (1, 50, 2000, 4, 2, 128, 64),
    (4, 100, 1500, 16, 4, 128, 64),  # chunks
])
def test_many_small_weights_beside_a_large_one(B, nq, ctx, hq, hk, d, group, size):
    page, g = 64, gen(96)
    pages = -(-ctx // page)
    cache = new_cache(pages, page, hk, d, group)
    k = normal(g, ctx, hk, d) * 0.25
    k[0] = 1.0
    off = torch.randn(1, hk, d, generator=g, device="cuda") * 2  # channels far from each other: sums do not average out
    v = ((torch.randn(ctx, hk, d, generator=g, device="cuda") * 0.3 + off) * size).bfloat16()
    v[0] = 0
    mbw.kv4_append(cache, k, v, torch.arange(ctx, device="cuda"))
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(B, 1)  # the same tokens for every request
    q = (torch.randn(B * nq, hq, d, generator=g, device="cuda") * 0.1 + 9.0 * d ** -0.5).bfloat16()
    c = torch.full((B,), ctx, dtype=torch.int32, device="cuda")
    (kn, ks, km), (vn, vs, vm) = ref.quantize(k, group), ref.quantize(v, group)
    kk, vv, mass = kn * ks + km, vn * vs + vm, (vs * (vn - 8)).abs() + (vm + 8 * vs).abs()
    x = torch.einsum("thd,qhgd->qhgt", kk, ref.f64(q).view(B * nq, hk, hq // hk, d)) * d ** -0.5
    pos = ctx - nq + torch.arange(B * nq) % nq
    x = x.masked_fill((torch.arange(ctx) > pos[:, None])[:, None, None], -float("inf"))
    p = x.softmax(-1)
    assert 0.3 < float(p[..., 0].min()) and float(p[..., 1:].max()) < 0.01
    want, tol = (torch.einsum("qhgt,thd->qhgd", p, y).reshape(B * nq, hq, d) for y in (vv, mass))
    for ws in (None, mbw.kv4_attention_workspace(d)):
        with mbw.output_fp32():
            out = ref.f64(mbw.kv4_attention(cache, q, table, c, workspace=ws))
        err = (out - want).abs()
        assert (err <= tol * 2.0 ** -10 + 2.0 ** -40 * size).all(), float((err / tol).max())
        out = ref.f64(mbw.kv4_attention(cache, q, table, c, workspace=ws))
        err = (out - want).abs()
        assert (err <= tol * 2.0 ** -10 + want.abs() * 2.0 ** -8 + 2.0 ** -40 * size).all(), float((err / tol).max())


@pytest.mark.parametrize("way", ["rising", "falling", "one large"])
@pytest.mark.parametrize("B,nq,hq,hk,d,group", [(64, 1, 16, 8, 128, 64), (1, 1, 4, 2, 64, 32), (40, 30, 8, 2, 256, 64), (2, 1, 2, 1, 256, 32)])
def test_scales_that_change_along_the_context(B, nq, hq, hk, d, group, way):
    page, ctx, g = 16, 1000, gen(97)
    cache = new_cache(-(-ctx // page), page, hk, d, group)
    power = torch.linspace(-16, 13, ctx, device="cuda")
    if way == "falling":
        power = power.flip(0)
    elif way == "one large":
        power[:] = -12
        power[ctx // 2] = 13
    k = normal(g, ctx, hk, d) * 0.25
    v = ((torch.randn(ctx, hk, d, generator=g, device="cuda") * 0.3 + 0.5) * power.round().exp2()[:, None, None]).bfloat16()
    mbw.kv4_append(cache, k, v, torch.arange(ctx, device="cuda"))
    table = torch.arange(-(-ctx // page), dtype=torch.int32, device="cuda").repeat(B, 1)
    q = normal(g, B * nq, hq, d)
    c = torch.full((B,), ctx, dtype=torch.int32, device="cuda")
    (kn, ks, km), (vn, vs, vm) = ref.quantize(k, group), ref.quantize(v, group)
    kk, vv, mass = kn * ks + km, vn * vs + vm, (vs * (vn - 8)).abs() + (vm + 8 * vs).abs()
    x = torch.einsum("thd,qhgd->qhgt", kk, ref.f64(q).view(B * nq, hk, hq // hk, d)) * d ** -0.5
    pos = ctx - nq + torch.arange(B * nq) % nq
    p = x.masked_fill((torch.arange(ctx) > pos[:, None])[:, None, None], -float("inf")).softmax(-1)
    want, tol = (torch.einsum("qhgt,thd->qhgd", p, y).reshape(B * nq, hq, d) for y in (vv, mass))
    for ws in (None, mbw.kv4_attention_workspace(d)):
        with mbw.output_fp32():
            out = ref.f64(mbw.kv4_attention(cache, q, table, c, workspace=ws))
        assert ((out - want).abs() <= tol * 2.0 ** -10).all(), float(((out - want).abs() / tol).max())


@pytest.mark.parametrize("fill", [0x7B, 0xFB, 0x6F, 0xFE, 0x7C, 0x00])
@pytest.mark.parametrize("B,nq,d,group", [(1, 1, 128, 64), (40, 1, 128, 32), (40, 3, 64, 64), (3, 20, 256, 64), (1, 2, 256, 32)])
def test_scales_of_tokens_that_no_query_sees_do_not_enter(fill, B, nq, d, group):
    """Tokens before every window were never appended; what their bytes say of their scales changes no bit."""
    hq, hk, ctx, first, page, window = 16, 2, 700, 627, 16, 40
    outs = []
    for byte in (fill, 0x31):
        g = gen(98)
        cache = new_cache(-(-ctx // page) + 1, page, hk, d, group, fill=byte)
        k, v, q = normal(g, ctx - first, hk, d), normal(g, ctx - first, hk, d) * 1e-3, normal(g, B * nq, hq, d)
        mbw.kv4_append(cache, k, v, torch.arange(first, ctx, device="cuda"))
        table = torch.arange(-(-ctx // page), dtype=torch.int32, device="cuda").repeat(B, 1)
        c = torch.full((B,), ctx - 5, dtype=torch.int32, device="cuda")  # its last page is not full
        outs.append([mbw.kv4_attention(cache, q, table, c, window=window, return_lse=True, workspace=ws)
                     for ws in (None, mbw.kv4_attention_workspace(d))])
    for (a, x), (b, y) in zip(*outs):
        assert a.isfinite().all() and torch.equal(a, b) and torch.equal(x, y)
