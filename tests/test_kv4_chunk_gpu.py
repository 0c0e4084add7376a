"""kv4_attention over chunks of a prompt (128 query rows per KV head and more), against its definition in 64 bits.

Tolerances count roundings. A score is off by what the rounding of s (n - 8) to fp16, 2^-11 of it, moves in q . k, and by
fp32 sums; a weight by its score and by its own rounding to fp16, 2^-11; values s (n - 8) by 2^-11; the result by its
rounding to bf16, 2^-8. Weights and their sum are rounded alike, so a weight's error acts on |v - out|.
"""
import pytest
import torch

import kv4_ref as ref
import memory_bound_weight_gb300 as mbw
from test_kv4_gpu import gen, new_cache, normal

pytestmark = pytest.mark.gpu


def cache_of(seed, ctx, page, hk, d, group, make):
    """A cache with each request's tokens from make(g, n) -> (k, v), the rest of it NaN; random pages, -1 past a request's
    last; and per request the codes, scales and minima of K and V in 64 bits."""
    g = gen(seed)
    used = [-(-c // page) for c in ctx]
    cache = new_cache(sum(used) + 2, page, hk, d, group)
    order = torch.randperm(sum(used) + 2, generator=g, device="cuda").cpu()
    table = torch.full((len(ctx), max(max(used), 1)), -1, dtype=torch.int32)
    at, kv = 0, []
    for b, c in enumerate(ctx):
        table[b, :used[b]] = order[at:at + used[b]]
        at += used[b]
        k, v = make(g, c)
        if c:
            t = torch.arange(c)
            mbw.kv4_append(cache, k, v, (table[b].long()[t // page] * page + t % page).cuda())
        kv.append((ref.quantize(k, group), ref.quantize(v, group)))
    return cache, table.cuda(), kv, g


def exact(q, kv, ctx, starts, scale, window):
    """out, lse, and the bounds on their errors before the last rounding."""
    q = ref.f64(q)
    T, hq, d = q.shape
    out, tol = torch.zeros(T, hq, d, dtype=torch.float64), torch.zeros(T, hq, d, dtype=torch.float64)
    lse, ltol = torch.full((T, hq), -float("inf"), dtype=torch.float64), torch.zeros(T, hq, dtype=torch.float64)
    for b, ((kn, ks, km), (vn, vs, vm)) in enumerate(kv):
        nq, n = starts[b + 1] - starts[b], ctx[b]
        if nq == 0 or n == 0:
            continue
        pos = torch.arange(n - nq, n)[:, None]
        t = torch.arange(n)[None]
        see = (t <= pos) & (t > pos - window if window else t >= 0)
        for h in range(hq):
            i, rows = h * ks.shape[1] // hq, slice(starts[b], starts[b + 1])
            k, kc = kn[:, i] * ks[:, i] + km[:, i], (ks[:, i] * (kn[:, i] - 8)).abs()
            v, vc = vn[:, i] * vs[:, i] + vm[:, i], (vs[:, i] * (vn[:, i] - 8)).abs()
            x = (q[rows, h] @ k.T * scale).masked_fill(~see, -float("inf"))
            off = (q[rows, h].abs() @ (kc * 2.0 ** -11 + k.abs() * 2.0 ** -20).T * abs(scale)).masked_fill(~see, 0).amax(1)
            none = ~see.any(1)
            p = torch.softmax(x, 1).masked_fill(none[:, None], 0)
            o = p @ v
            lse[rows, h] = torch.logsumexp(x, 1)
            ltol[rows, h] = off + 2.0 ** -11 + x.masked_fill(~see, 0).abs().amax(1) * 2.0 ** -20
            e = (ltol[rows, h] * (1 + 2.0 ** -4))[:, None]
            away = torch.stack([(p[:, :, None] * (v[None, :, c:c + 8] - o[:, None, c:c + 8]).abs()).sum(1) for c in range(0, d, 8)], 1)
            out[rows, h] = o
            tol[rows, h] = e * away.reshape(-1, d) + p @ vc * 2.0 ** -11 * (1 + 2.0 ** -4) + p @ v.abs() * 2.0 ** -20 + 2.0 ** -40
    return out, lse, tol, ltol


def run(cache, q, table, ctx, starts, **kw):
    c, s = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (ctx, starts))
    return mbw.kv4_attention(cache, q, table, c, s, return_lse=True, **kw)


def check(got, want):
    out, lse, tol, ltol = want
    o, l = ref.f64(got[0]), ref.f64(got[1])
    half = 0 if got[0].dtype == torch.float32 else 2.0 ** -8 * (1 + 2.0 ** -6)
    err, bound = (o - out).abs(), tol * (1 + half) + out.abs() * half + 2.0 ** -134
    assert (err <= bound).all(), (float(err.max()), float((err / bound).max()))
    none = lse == -float("inf")
    assert (l[none] == -float("inf")).all()
    assert ((l - lse).abs()[~none] <= (ltol + lse.abs() * 2.0 ** -22)[~none]).all(), float((l - lse).abs()[~none].max())


def starts_of(nq):
    s = [0]
    for n in nq:
        s.append(s[-1] + n)
    return s


CASES = [
    # ctx, queries per request, hq, hk, d, group, page, window
    ([300], [300], 8, 2, 128, 64, 16, 0),
    ([128], [128], 1, 1, 128, 64, 128, 0),
    ([90, 700, 1], [70, 133, 0], 32, 8, 128, 64, 32, 20),
    ([1000, 129], [200, 128], 28, 4, 128, 32, 64, 0),
    ([130], [130], 32, 4, 64, 32, 16, 0),
    ([513, 50], [100, 50], 16, 4, 64, 64, 16, 100),
    ([3, 12, 400], [5, 12, 200], 8, 1, 128, 64, 16, 0),
    ([2000], [64], 16, 1, 128, 64, 48, 0),
    ([4100], [33], 20, 4, 64, 64, 1024, 3000),
    ([140, 90, 260, 200] * 20, [100, 90, 1, 160] * 20, 4, 2, 128, 64, 16, 0),
    ([40, 300], [33, 100], 7, 1, 128, 32, 16, 1),
    ([2000], [64], 32, 2, 128, 64, 48, 0),
    ([4100, 1500], [33, 40], 32, 4, 64, 64, 1024, 3000),
    ([1300, 0, 2600], [40, 3, 55], 48, 4, 128, 32, 16, 0),
    ([1, 130, 1100] * 14, [1, 120, 50] * 14, 8, 2, 64, 32, 16, 0),
]


@pytest.mark.parametrize("i", range(len(CASES)))
@pytest.mark.parametrize("space", ["full", "none"])
def test_chunks(i, space):
    ctx, nq, hq, hk, d, group, page, window = CASES[i]
    cache, table, kv, g = cache_of(i, ctx, page, hk, d, group,
                                   lambda g, n: (normal(g, n, hk, d) + normal(g, 1, hk, d) * 3, normal(g, n, hk, d) + 0.3))
    starts = starts_of(nq)
    q = normal(g, starts[-1], hq + 3, d)[:, :hq]
    ws = mbw.kv4_attention_workspace(d) if space == "full" else None
    want = exact(q, kv, ctx, starts, d ** -0.5, window)
    got = run(cache, q, table, ctx, starts, window=window, workspace=ws)
    check(got, want)
    again = run(cache, q, table, ctx, starts, window=window, workspace=ws)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])  # bitwise, run after run
    with mbw.output_fp32():
        check(run(cache, q, table, ctx, starts, window=window, workspace=ws), want)


@pytest.mark.parametrize("scale", [-0.25, 0.0, 2.0])
@pytest.mark.parametrize("size", [2.0 ** -18, 1.0, 2.0 ** 12])
def test_chunk_scales_and_sizes_of_queries(scale, size):
    """Scores of up to some hundred, where one key takes all, and queries far from 1; a maximum that grows on the way."""
    ctx, nq, hq, hk, d = [400, 150], [140, 150], 8, 2, 128
    grow = torch.linspace(0.2, 3, 400, device="cuda")
    cache, table, kv, g = cache_of(60, ctx, 16, hk, d, 64, lambda g, n: ((normal(g, n, hk, d) * grow[:n, None, None]).bfloat16(), normal(g, n, hk, d)))
    q = (normal(g, sum(nq), hq, d) * size).bfloat16()
    want = exact(q, kv, ctx, starts_of(nq), scale / size, 0)
    check(run(cache, q, table, ctx, starts_of(nq), scale=scale / size, workspace=mbw.kv4_attention_workspace(d)), want)


@pytest.mark.parametrize("size", [2.0 ** -20, 65000.0])
def test_chunk_values_at_the_ends_of_their_range(size):
    """Scales beyond 8188, whose 8 steps pass fp16, and scales that are fp16 subnormals."""
    ctx, nq, hq, hk, d = [200], [140], 16, 2, 64
    cache, table, kv, g = cache_of(61, ctx, 16, hk, d, 32, lambda g, n: (
        (normal(g, n, hk, d).clamp(-1, 1) * size).bfloat16(), (normal(g, n, hk, d).clamp(-1, 1) * size).bfloat16()))
    assert size < 1 or float(kv[0][1][1].max()) > 8188
    q = normal(g, sum(nq), hq, d)
    want = exact(q, kv, ctx, starts_of(nq), 1 / size / 8, 0)
    with mbw.output_fp32():
        check(run(cache, q, table, ctx, starts_of(nq), scale=1 / size / 8), want)


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("space", ["full", "none"])
def test_chunk_nan_reaches_the_queries_that_see_it_alone(which, space):
    ctx, nq, hq, hk, d, at, group = [300, 260], [150, 150], 8, 2, 128, 230, 64

    def make(g, n):
        return [normal(g, n, hk, d), normal(g, n, hk, d)]

    cache, table, kv, g = cache_of(62, ctx, 16, hk, d, group, make)
    k, v = normal(g, 1, hk, d), normal(g, 1, hk, d)
    (k if which == "k" else v)[0, 1, 70] = float("nan")  # group 1 of KV head 1 of request 0's token `at`
    mbw.kv4_append(cache, k, v, (table[0, at // 16].long() * 16 + at % 16).reshape(1).cuda())
    for x, (n, s, m) in zip((k, v), kv[0]):
        for to, new in zip((n, s, m), ref.quantize(x, group)):
            to[at] = new[0]
    q = normal(g, sum(nq), hq, d)
    ws = mbw.kv4_attention_workspace(d) if space == "full" else None
    for window in (0, 40):
        out, lse = run(cache, q, table, ctx, starts_of(nq), window=window, workspace=ws)
        pos = torch.cat([torch.arange(c - n, c) for c, n in zip(ctx, nq)])
        hit = (torch.arange(sum(nq)) < nq[0]) & (pos >= at) & ((pos - window < at) if window else pos >= 0)
        bad = torch.zeros(sum(nq), hq, d, dtype=torch.bool)
        bad[hit, 4:, (0 if which == "k" else 64):] = True
        assert torch.equal(torch.isnan(ref.f64(out)), bad)
        want = exact(q, [[tuple(x.nan_to_num(0) for x in y) for y in z] for z in kv], ctx, starts_of(nq), d ** -0.5, window)
        clean = ~bad
        if which == "k":
            assert torch.equal(torch.isnan(ref.f64(lse)), bad.any(2))
            for i in (0, 1):
                want[i][bad if i == 0 else bad.any(2)] = 0
        err = ((ref.f64(out) - want[0]).abs() - (want[2] * (1 + 2.0 ** -8) + want[0].abs() * (2.0 ** -8 + 2.0 ** -14)))[clean]
        assert (err <= 0).all(), float(err.max())


def test_chunks_of_more_requests_than_threads():
    hq, hk, d, B = 16, 1, 64, 950
    ctx, nq = [(11 * i) % 37 + 7 for i in range(B)], [5 + i % 3 for i in range(B)]
    cache, table, kv, g = cache_of(65, ctx, 16, hk, d, 64, lambda g, n: (normal(g, n, hk, d), normal(g, n, hk, d)))
    starts = starts_of(nq)
    q = normal(g, starts[-1], hq, d)
    check(run(cache, q, table, ctx, starts, scale=0.1), exact(q, kv, ctx, starts, 0.1, 0))


def test_chunk_page_or_length_out_of_range_is_reported():
    ctx, nq, hq, hk, d = [200, 180], [150, 150], 8, 1, 64
    cache, table, kv, g = cache_of(63, ctx, 16, hk, d, 64, lambda g, n: (normal(g, n, hk, d), normal(g, n, hk, d)))
    q = normal(g, sum(nq), hq, d)
    run(cache, q, table, ctx, starts_of(nq))
    mbw.check_device_error()
    table[0, 3] = 10 ** 6
    run(cache, q, table, ctx, starts_of(nq))
    with pytest.raises(mbw.MbwError):
        mbw.check_device_error()
    table[0, 3] = 0
    run(cache, q, table, [10 ** 7, 180], starts_of(nq))
    with pytest.raises(mbw.MbwError):
        mbw.check_device_error()
    mbw.check_device_error()


def test_chunk_in_a_graph_follows_the_lengths():
    ctx, nq, hq, hk, d = [600, 300], [64, 64], 16, 2, 128
    cache, table, kv, g = cache_of(64, ctx, 16, hk, d, 64, lambda g, n: (normal(g, n, hk, d), normal(g, n, hk, d)))
    q = normal(g, sum(nq), hq, d)
    c = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    s = torch.tensor(starts_of(nq), dtype=torch.int32, device="cuda")
    ws = mbw.kv4_attention_workspace(d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mbw.kv4_attention(cache, q, table, c, s, workspace=ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = mbw.kv4_attention(cache, q, table, c, s, workspace=ws)
    torch.cuda.synchronize()
    for lens in (ctx, [200, 299], [64, 130], [600, 300]):
        c.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        cut = [[tuple(x[:n] for x in y) for y in z] for z, n in zip(kv, lens)]
        want = exact(q, cut, lens, starts_of(nq), d ** -0.5, 0)
        bound = want[2] * (1 + 2.0 ** -8) + want[0].abs() * (2.0 ** -8 + 2.0 ** -14)
        assert ((ref.f64(out) - want[0]).abs() <= bound).all()
