"""kv4_attention_shared, against the definition of attention in 64 bits and against kv4_attention. The bounds are those of
tests/test_kv4_chunk_gpu.py, whose kernel computes the shared part: the other part's are within them, and the parts' join
is a product and a sum in fp32 each."""
import pytest
import torch

import kv4_ref as ref
import memory_bound_weight_gb300 as mbw
from test_kv4_chunk_gpu import check, exact, starts_of
from test_kv4_gpu import gen, new_cache, normal

pytestmark = pytest.mark.gpu


def shared_cache(seed, prefix, ctx, page, hk, d, group, make=None, keep=None):
    """A cache whose requests begin with the same `prefix` tokens, in whole pages the same ones, the rest of it NaN; -1 in
    the block table past a request's last page. Per request (of those in `keep`) the codes, scales and minima of its K and V."""
    g = gen(seed)
    make = make or (lambda g, n: (normal(g, n, hk, d) + normal(g, 1, hk, d) * 2, normal(g, n, hk, d) + 0.3))
    common = prefix // page
    used = [-(-c // page) for c in ctx]
    own = [max(0, u - common) for u in used]
    total = common + sum(own) + 2
    cache = new_cache(total, page, hk, d, group)
    order = torch.randperm(total, generator=g, device="cuda").cpu()
    table = torch.full((len(ctx), max(max(used), common, 1)), -1, dtype=torch.int32)
    longest, at, kv = max(ctx), common, []
    kp, vp = make(g, max(prefix, 1))
    for b, c in enumerate(ctx):
        table[b, :min(used[b], common)] = order[:min(used[b], common)]
        table[b, common:common + own[b]] = order[at:at + own[b]]
        at += own[b]
        ko, vo = make(g, max(c - prefix, 1))
        k, v = torch.cat((kp[:c], ko[:max(0, c - prefix)])), torch.cat((vp[:c], vo[:max(0, c - prefix)]))
        if c:
            t = torch.arange(c)
            slots = table[b].long()[t // page] * page + t % page
            slots[:min(c, common * page)] = slots[:min(c, common * page)] if c == longest else -1  # shared pages written once
            mbw.kv4_append(cache, k, v, slots.cuda())
        kv.append((ref.quantize(k, group), ref.quantize(v, group)) if keep is None or b in keep else None)
    return cache, table.cuda(), kv, g


def run(cache, q, table, ctx, starts, prefix, **kw):
    c = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    s = None if starts is None else torch.tensor(starts, dtype=torch.int32, device="cuda")
    return mbw.kv4_attention_shared(cache, q, table, c, prefix, s, return_lse=True, **kw)


# The shared part has a kernel of its own where reading the shared pages for every request would take longer: long prefixes of
# many requests. What decides is a bound on the time, so that the cases below are on one side or the other by a factor.
LARGE = [
    # prefix, ctx, queries per request, hq, hk, d, group, page, window
    (3000, [3001 + 7 * i for i in range(64)], [1] * 64, 32, 8, 128, 64, 32, 0),
    (9000, [9040, 9200, 9007, 9001], [8, 5, 8, 8], 28, 4, 128, 32, 64, 0),                              # few requests: CTAs as workers behind it
    (1500, [1500 + (37 * i) % 90 - 20 for i in range(200)], [1] * 200, 32, 8, 64, 32, 16, 0),            # some end inside the prefix
    (1530, [1700, 0, 1531, 90, 1600, 1, 0, 3] * 16, [4, 1, 8, 1, 0, 5, 0, 8] * 16, 16, 4, 128, 64, 16, 0),  # padding, one token, no queries, more queries than tokens
    (2048, [0, 0] + [2100, 2048, 2049, 0] * 25, [1, 2] + [3, 4, 1, 1] * 25, 32, 8, 64, 64, 32, 0),         # the first rows are padding; lengths that end with the prefix
    (2000, [1900, 300, 17, 1024, 16] * 16, [1, 3, 8, 8, 8] * 16, 32, 8, 128, 64, 16, 0),                   # all inside the prefix
    (2500, [2600, 2501, 2900] * 30, [2, 4, 8] * 30, 32, 8, 128, 64, 16, 200),                              # windows that leave one, none or most of it behind
    (2500, [2600, 2501, 2900] * 30, [2, 4, 8] * 30, 32, 8, 64, 64, 48, 1700),
    (2500, [2600, 2501, 2900] * 30, [2, 4, 8] * 30, 32, 8, 128, 32, 16, 1),
    (9216, [9220 + 11 * i for i in range(130)], [1] * 130, 4, 1, 128, 64, 1024, 0),
    (3111, [3150 + (i * 29) % 500 for i in range(40)], [11] * 40, 8, 1, 128, 32, 16, 0),                   # a row tile's end within a query
    (777, [800 + i % 9 for i in range(250)], [1 + i % 5 for i in range(250)], 20, 4, 128, 64, 16, 0),      # more items than SMs
    (125, [120 + i % 40 for i in range(400)], [8] * 400, 32, 8, 128, 64, 16, 0),                            # 112 shared tokens, less than a tile
]

CASES = LARGE + [
    (256, [300, 257, 400, 280], [1] * 4, 8, 2, 128, 64, 16, 0),
    (1000, [1001, 1030, 1100], [1] * 3, 28, 4, 128, 64, 64, 0),
    (128, [129], [1], 1, 1, 64, 64, 16, 0),
    (2000, [2001 + 7 * i for i in range(64)], [1] * 64, 32, 8, 128, 64, 32, 0),
    (700, [700 + 3 + i % 50 for i in range(130)], [1] * 130, 32, 4, 64, 32, 16, 0),
    (3000, [3040, 3200, 3007], [2, 5, 3], 28, 4, 128, 32, 64, 0),
    (530, [700, 0, 531, 90, 600], [1, 1, 1, 1, 0], 8, 2, 128, 64, 16, 0),   # padding, one inside the prefix, one without queries
    (512, [0, 0, 530, 512, 513], [1, 2, 3, 4, 1], 16, 4, 64, 64, 32, 0),    # the first rows are padding; lengths that end with the prefix
    (640, [100, 300, 17], [1, 3, 17], 8, 8, 128, 64, 16, 0),                # all inside the prefix
    (1500, [1600, 1501, 1900], [1, 2, 1], 8, 2, 128, 64, 16, 200),          # windows that leave one, none and all of the prefix behind
    (1500, [1600, 1501, 1900], [1, 2, 1], 8, 2, 64, 64, 48, 1000),
    (1500, [1600, 1501, 1900], [1, 2, 1], 8, 2, 128, 32, 16, 1),
    (1500, [1550, 1700], [40, 60], 16, 4, 128, 64, 16, 700),                # more queries than a tile has rows
    (900, [950, 1000, 901], [30, 7, 1], 16, 2, 256, 64, 16, 0),
    (900, [950 + i for i in range(20)], [1] * 20, 16, 8, 256, 32, 32, 0),
    (2048, [2100 + 11 * i for i in range(200)], [1] * 200, 4, 1, 128, 64, 1024, 0),
    (5000, [5003, 5001], [1, 1], 5, 5, 128, 64, 16, 0),
    (15, [40, 33], [1, 1], 8, 2, 128, 64, 16, 0),                            # no whole page
]


@pytest.mark.parametrize("i", range(len(CASES)))
def test_shared(i):
    prefix, ctx, nq, hq, hk, d, group, page, window = CASES[i]
    cache, table, kv, g = shared_cache(i, prefix, ctx, page, hk, d, group)
    starts = starts_of(nq)
    q = normal(g, starts[-1], hq + 3, d)[:, :hq]
    want = exact(q, kv, ctx, starts, d ** -0.5, window)
    s = None if set(nq) == {1} else starts
    ws = mbw.kv4_attention_shared_workspace(d, starts[-1], hq)
    n = mbw.launch_count()
    got = run(cache, q, table, ctx, s, prefix, window=window, workspace=ws)
    if i < len(LARGE):
        assert mbw.launch_count() == n + 2
    check(got, want)
    again = run(cache, q, table, ctx, s, prefix, window=window, workspace=ws)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])  # bitwise, and the workspace is as it was
    check(run(cache, q, table, ctx, s, prefix, window=window), want)  # no workspace
    small = mbw.kv4_attention_workspace(d)
    check(run(cache, q, table, ctx, s, prefix, window=window, workspace=small), want)
    with mbw.output_fp32():
        check(run(cache, q, table, ctx, s, prefix, window=window, workspace=ws), want)
    # the workspace serves the plain call too
    c = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    st = None if s is None else torch.tensor(s, dtype=torch.int32, device="cuda")
    check(mbw.kv4_attention(cache, q, table, c, st, window=window, workspace=ws, return_lse=True), want)
    # into rows of a wider output; the others keep what they hold
    wide = torch.full((starts[-1] + 1, hq + 1, d), 7.0, dtype=torch.bfloat16, device="cuda")
    mbw.kv4_attention_shared(cache, q, table, c, prefix, st, window=window, workspace=ws, out=wide[:-1, :hq])
    assert torch.equal(wide[:-1, :hq], got[0]) and wide[-1].eq(7).all() and wide[:, hq].eq(7).all()


def two_kernels(call):
    """The call's result, and that the shared part had its kernel."""
    n = mbw.launch_count()
    out = call()
    assert mbw.launch_count() == n + 2
    return out


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("d,group", [(64, 64), (64, 32), (128, 64), (256, 64)])
def test_nan_in_the_prefix_reaches_the_queries_that_see_it_alone(which, d, group):
    prefix, ctx, nq, hq, hk, at = 2320, [2340, 2400, 2250, 2360] * 100, [1, 2, 8, 5] * 100, 8, 2, 2290
    cache, table, _, g = shared_cache(70, prefix, ctx, 16, hk, d, group, keep=())
    k, v = normal(g, 1, hk, d), normal(g, 1, hk, d)
    (k if which == "k" else v)[0, 1, d - 1] = float("nan")  # the last group of KV head 1
    mbw.kv4_append(cache, k, v, (table[1, at // 16].long() * 16 + at % 16).reshape(1).cuda())
    starts = starts_of(nq)
    q = normal(g, starts[-1], hq, d)
    ws = mbw.kv4_attention_shared_workspace(d, starts[-1], hq)
    pos = torch.cat([torch.arange(c - n, c) for c, n in zip(ctx, nq)])
    for window in (0, 60):
        call = lambda: run(cache, q, table, ctx, starts, prefix, window=window, workspace=ws)  # noqa: E731
        out, lse = two_kernels(call) if d < 256 else call()
        hit = (pos >= at) & ((pos - window < at) if window else pos >= 0)
        bad = torch.zeros(starts[-1], hq, d, dtype=torch.bool)
        bad[hit, 4:, (0 if which == "k" else d - group):] = True
        assert torch.equal(torch.isnan(ref.f64(out)), bad)
        if which == "k":
            assert torch.equal(torch.isnan(ref.f64(lse)), bad.any(2))


@pytest.mark.parametrize("size", [2.0 ** -20, 60000.0])
def test_values_at_the_ends_of_their_range(size):
    prefix, ctx, hq, hk, d = 4400, [4420, 4500, 4401] * 30, 32, 8, 64
    cache, table, kv, g = shared_cache(71, prefix, ctx, 16, hk, d, 32, lambda g, n: (
        (normal(g, n, hk, d).clamp(-1, 1) * size).bfloat16(), (normal(g, n, hk, d).clamp(-1, 1) * size).bfloat16()))
    starts = starts_of([2] * 90)
    q = normal(g, 180, hq, d)
    want = exact(q, kv, ctx, starts, 1 / size / 8, 0)
    ws = mbw.kv4_attention_shared_workspace(d, 180, hq)
    with mbw.output_fp32():
        check(two_kernels(lambda: run(cache, q, table, ctx, starts, prefix, scale=1 / size / 8, workspace=ws)), want)


@pytest.mark.parametrize("far", [-3000.0, 0.0, 3000.0])
def test_scores_of_the_two_parts_far_apart(far):
    """The prefix's scores are some 10^3 below, beside or above the own tokens', with either sign of the scale."""
    prefix, ctx, hq, hk, d = 4256, [4300, 4280] * 20, 16, 8, 128
    first = []

    def make(g, n):
        k = normal(g, n, hk, d)
        if not first:
            first.append(1)
            k[..., 0] += far
        return k.bfloat16(), normal(g, n, hk, d)

    cache, table, kv, g = shared_cache(72, prefix, ctx, 16, hk, d, 32, make)
    starts = starts_of([4] * 40)
    q = normal(g, 160, hq, d)
    q[..., 0] = 1.0
    ws = mbw.kv4_attention_shared_workspace(d, 160, hq)
    for scale in (1.0, -1.0, 0.0):
        got = two_kernels(lambda: run(cache, q, table, ctx, starts, prefix, scale=scale, workspace=ws))
        check(got, exact(q, kv, ctx, starts, scale, 0))


def test_more_requests_than_threads():
    hq, hk, d, B, prefix = 16, 4, 128, 950, 400
    ctx = [prefix + (11 * i) % 37 - 5 for i in range(B)]
    nq = [i % 3 for i in range(B)]
    some = [i for i in range(B) if i % 40 in (5, 19)] + [B - 1]
    cache, table, kv, g = shared_cache(73, prefix, ctx, 16, hk, d, 64, keep=set(some))
    starts = starts_of(nq)
    q = normal(g, starts[-1], hq, d)
    ws = mbw.kv4_attention_shared_workspace(d, starts[-1], hq)
    out, lse = two_kernels(lambda: run(cache, q, table, ctx, starts, prefix, workspace=ws))
    rows = torch.cat([torch.arange(starts[i], starts[i + 1]) for i in some]).cuda()
    want = exact(q[rows], [kv[i] for i in some], [ctx[i] for i in some], starts_of([nq[i] for i in some]), d ** -0.5, 0)
    check((out[rows], lse[rows]), want)


def test_in_a_graph_follows_the_lengths():
    prefix, B, hq, hk, d = 3512, 48, 32, 8, 128
    ctx = [3600, 3530, 3700, 3513] * 12
    cache, table, kv, g = shared_cache(74, prefix, ctx, 16, hk, d, 64)
    q = normal(g, B, hq, d)
    c = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    ws = mbw.kv4_attention_shared_workspace(d, B, hq)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        two_kernels(lambda: mbw.kv4_attention_shared(cache, q, table, c, prefix, workspace=ws))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out, lse = mbw.kv4_attention_shared(cache, q, table, c, prefix, return_lse=True, workspace=ws)
    torch.cuda.synchronize()
    for lens in (ctx, [3520, 3530, 3513, 0] * 12, [100, 3512, 1, 400] * 12, [0] * B, ctx):
        c.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        cut = [[tuple(x[:n] for x in y) for y in z] for z, n in zip(kv, lens)]
        check((out, lse), exact(q, cut, lens, starts_of([1] * B), d ** -0.5, 0))


def test_what_comes_before_and_behind_on_the_stream():
    """The other tokens' kernel starts before the shared part's ends: it reads what was written in front of both, and what
    follows on the stream changes nothing under them."""
    prefix, hq, hk, d, B = 4032, 32, 8, 128, 40
    ctx = [4040 + 9 * i for i in range(B)]
    cache, table, kv, g = shared_cache(75, prefix, ctx, 16, hk, d, 64, keep=())
    qs = [normal(g, B, hq, d) for _ in range(6)]
    c = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    ws = mbw.kv4_attention_shared_workspace(d, B, hq)
    want = [mbw.kv4_attention_shared(cache, q, table, c, prefix, workspace=ws) for q in qs]
    buf, out = torch.empty_like(qs[0]), torch.empty_like(qs[0])
    torch.cuda.synchronize()
    got = []
    for _ in range(4):
        for q in qs:
            buf.copy_(q)
            mbw.kv4_attention_shared(cache, buf, table, c, prefix, workspace=ws, out=out)
            buf.fill_(float("nan"))
            got.append(out.clone())
            out.zero_()
    torch.cuda.synchronize()
    assert all(torch.equal(x, want[i % 6]) for i, x in enumerate(got))


def test_two_streams_with_their_own_workspaces():
    prefix, hq, hk, d = 4032, 32, 8, 128
    ctx = [4040 + 9 * i for i in range(40)]
    cache, table, kv, g = shared_cache(75, prefix, ctx, 16, hk, d, 64, keep=())
    q = [normal(g, 40, hq, d) for _ in range(2)]
    c = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    ws = [mbw.kv4_attention_shared_workspace(d, 40, hq) for _ in range(2)]
    want = [two_kernels(lambda: mbw.kv4_attention_shared(cache, q[i], table, c, prefix, workspace=ws[i])) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(mbw.kv4_attention_shared(cache, q[i], table, c, prefix, workspace=ws[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, want[i]) for x in got[i])


def test_pages_lengths_and_offsets_out_of_range_are_reported():
    prefix, hq, hk, d, B = 6128, 16, 8, 64, 60
    ctx = [6200, 6180, 6150] * 20
    cache, table, _, g = shared_cache(76, prefix, ctx, 16, hk, d, 64, keep=())
    q = normal(g, 2 * B, hq, d)
    ws = mbw.kv4_attention_shared_workspace(d, 2 * B, hq)
    ok = starts_of([2] * B)
    good = two_kernels(lambda: run(cache, q, table, ctx, ok, prefix, workspace=ws))
    mbw.check_device_error()
    for row, entry in ((0, 3), (2, 384)):  # of the prefix (the longest request's row), of a request's own
        keep = int(table[row, entry])
        table[row, entry] = 10 ** 6
        run(cache, q, table, ctx, ok, prefix, workspace=ws)
        with pytest.raises(mbw.MbwError):
            mbw.check_device_error()
        table[row, entry] = keep
    falls, past, before = ok[:], ok[:], ok[:]
    falls[5], past[-1], before[0] = 40, 2 * B + 6, -1
    for starts, lens in ((ok, [10 ** 7] + ctx[1:]), (falls, ctx), (past, ctx), (before, ctx)):
        run(cache, q, table, lens, starts, prefix, workspace=ws)
        with pytest.raises(mbw.MbwError):
            mbw.check_device_error()
    again = run(cache, q, table, ctx, ok, prefix, workspace=ws)  # the workspace was left ready
    assert torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])
    mbw.check_device_error()
