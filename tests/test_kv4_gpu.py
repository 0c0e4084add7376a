"""The 4-bit paged cache on the GPU: appending with rotation, reading back, and
attention over it, against plain forms in 64 bits."""
import pytest

import kv4_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - the marker keeps these off CPU runs
    pytest.skip("needs a GPU", allow_module_level=True)

import memory_bound_weight_gb300 as mbw  # noqa: E402
from memory_bound_weight_gb300 import _binding as B  # noqa: E402

NAN_HALF = 0x7E00


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda").bfloat16()


def new_cache(num_pages, page, hk, d, group, fill=0xFE):
    """A cache whose bytes all hold `fill`: 0xFEFE is a NaN in fp16, so that whatever was not written shows."""
    pages = torch.full((num_pages, mbw.kv4_page_bytes(page, hk, d, group)), fill, dtype=torch.uint8, device="cuda")
    return mbw.Kv4Cache(pages, hk, d, page, group)


def ulp_bf16(x):
    return x.abs() * 2.0 ** -8 + 2.0 ** -133


# ------------------------------------------------------------------ append ----
@pytest.mark.parametrize("T,hq,hk,d,group,page,rotary,inter", [
    (1, 28, 4, 128, 64, 16, 128, False), (1, 1, 1, 64, 32, 16, 64, True), (2, 32, 4, 64, 64, 32, 32, False),
    (5, 32, 8, 128, 32, 16, 64, True), (17, 16, 8, 256, 64, 64, 256, False), (33, 5, 5, 256, 32, 48, 16, True),
    (130, 7, 1, 128, 64, 128, 96, False), (700, 28, 4, 128, 64, 64, 128, False), (64, 0, 3, 64, 32, 16, 48, False),
    (9, 4, 2, 128, 64, 1024, 0, False), (300, 32, 8, 128, 32, 32, 112, True),
])
def test_append_then_gather(T, hq, hk, d, group, page, rotary, inter):
    g = gen(T * 1000 + d)
    wide = normal(g, T, (hq + 2 * hk) * d + 8)[:, 8:]  # rows of a wider matrix, 16 bytes past its start
    wide = wide.view(T, hq + 2 * hk, d) if T == 1 else wide.unflatten(1, (hq + 2 * hk, d))
    q, k, v = wide[:, :hq], wide[:, hq:hq + hk], wide[:, hq + hk:]
    num = -(-T // page) + 2
    cache = new_cache(num, page, hk, d, group)
    before = cache.pages.clone()
    slots = torch.randperm(num * page, generator=g, device="cuda")[:T]
    if T > 4:
        slots[torch.randperm(T, generator=g, device="cuda")[:T // 5]] = -1
    kw, pos, table = {}, None, None
    if rotary:
        table = mbw.rope_table(5000, rotary, 1e6)
        pos = torch.randint(5000, (T,), generator=g, device="cuda").to(torch.int32)
        kw = {"positions": pos, "cos_sin": table, "interleaved": inter}
    out = mbw.kv4_append(cache, k, v, slots, q=q if hq else None, **kw)
    kk, vv = mbw.kv4_gather(cache, slots)
    kr = ref.rotate(k, table, pos, inter) if rotary else ref.f64(k)
    kn, ks, km = ref.quantize(kr.float().bfloat16(), group)
    vn, vs, vm = ref.quantize(v, group)
    there = (slots >= 0).cpu()[:, None, None]
    # codes, scales and minima are functions of the inputs alone; s n + m is one fma in fp32, then rounded to bf16
    for got, (n, s, m) in ((kk, (kn, ks, km)), (vv, (vn, vs, vm))):
        want = torch.where(there, n * s + m, 0.0)
        err = (ref.f64(got) - want).abs()
        assert (err <= ulp_bf16(want) * (1 + 2.0 ** -10)).all(), float(err.max())
    if hq:
        want = ref.rotate(q, table, pos, inter) if rotary else ref.f64(q)
        assert (ref.f64(out) - want).abs().le(ulp_bf16(want) * (1 + 2.0 ** -10)).all()
        if not rotary:
            assert torch.equal(out, q)
    else:
        assert out is None
    # the other tokens' values: still NaN (their bytes are whole words of their own)
    free = torch.ones(num * page, dtype=torch.bool, device="cuda")
    free[slots[slots >= 0]] = False
    rest = free.nonzero()[:, 0]
    k0, v0 = mbw.kv4_gather(cache, rest)
    assert k0.isnan().all() and v0.isnan().all()
    # written again with nothing to store, nothing changes
    now = cache.pages.clone()
    mbw.kv4_append(cache, k, v, torch.full_like(slots, -1))
    assert torch.equal(cache.pages, now)
    if not there.any():
        assert torch.equal(now, before)


def test_append_rotates_queries_in_place():
    g = gen(3)
    wide = normal(g, 40, 12, 128)
    q, k, v = wide[:, :8], wide[:, 8:10], wide[:, 10:]
    table, pos = mbw.rope_table(64, 128), torch.arange(40, dtype=torch.int32, device="cuda")
    want = ref.rotate(q, table, pos, False)
    keep = wide[:, 8:].clone()
    cache = new_cache(3, 16, 2, 128, 64)
    out = mbw.kv4_append(cache, k, v, torch.arange(40, device="cuda"), q=q, positions=pos, cos_sin=table, q_out=q)
    assert out is q and (ref.f64(q) - want).abs().le(ulp_bf16(want) * (1 + 2.0 ** -10)).all()
    assert torch.equal(wide[:, 8:], keep)


def test_append_groups_that_are_flat_tiny_huge_or_not_numbers():
    d, group = 128, 64
    x = torch.zeros(9, 1, d, device="cuda")
    x[1] = 2.5  # one value: scale 0
    x[2, 0, 3] = 2.0 ** -30  # range below fp16
    x[3] = torch.linspace(-60000, 60000, d, device="cuda")
    x[4, 0, 5] = float("nan")
    x[5, 0, 70] = float("inf")
    x[6, 0, 70] = -1e30
    x[7] = -torch.linspace(1, 2, d, device="cuda") * 1e-3
    x[8, 0, :64], x[8, 0, 64:] = 3.0e38, -0.0
    x = x.bfloat16()
    cache = new_cache(1, 16, 1, d, group)
    slots = torch.arange(9, device="cuda")
    mbw.kv4_append(cache, x, x, slots)
    k, v = (ref.f64(t)[:, 0] for t in mbw.kv4_gather(cache, slots))
    n, s, m = (t[:, 0] for t in ref.quantize(x, group))
    want = n * s + m
    for got in (k, v):
        assert got[4, :64].isnan().all() and got[5, 64:].isnan().all() and got[6, 64:].isnan().all()
        assert got[8, :64].isnan().all() and got[8, 64:].eq(0).all()
        assert got[1].eq(2.5).all() and got[0].eq(0).all()
        for row, cols in ((2, slice(0, d)), (3, slice(0, d)), (4, slice(64, d)), (5, slice(0, 64)), (6, slice(0, 64)),
                          (7, slice(0, d))):
            assert (got[row, cols] - want[row, cols]).abs().le(ulp_bf16(want[row, cols]) * (1 + 2.0 ** -10)).all(), row


def test_slot_and_position_out_of_range_are_reported_and_not_stored():
    cache = new_cache(2, 16, 1, 64, 32)
    x = normal(gen(1), 3, 1, 64)
    before = cache.pages.clone()
    mbw.kv4_append(cache, x, x, torch.tensor([32, 1 << 40, 33], device="cuda"))
    assert torch.equal(cache.pages, before)
    with pytest.raises(mbw.MbwError) as e:
        mbw.check_device_error()
    assert e.value.status == 8
    k, _ = mbw.kv4_gather(cache, torch.tensor([32, 5000], device="cuda"))
    assert k.eq(0).all()
    with pytest.raises(mbw.MbwError):
        mbw.check_device_error()
    mbw.kv4_append(cache, x, x, torch.arange(3, device="cuda"), positions=torch.tensor([0, 9, -1], dtype=torch.int32,
                   device="cuda"), cos_sin=mbw.rope_table(9, 64))
    with pytest.raises(mbw.MbwError):
        mbw.check_device_error()
    mbw.check_device_error()


# --------------------------------------------------------------- attention ----
def filled(seed, ctx, page, hk, d, group, spare=2, spread=1.0, num_pages=None):
    """A cache in which each request's tokens are written and the rest is NaN, its block table (random pages; -1
    past a request's last), and the values it holds, in 64 bits."""
    g = gen(seed)
    used = [-(-c // page) for c in ctx]
    num = num_pages or sum(used) + spare
    cache = new_cache(num, page, hk, d, group)
    order = torch.randperm(sum(used) + spare, generator=g, device="cuda").cpu() + (num - sum(used) - spare)
    table = torch.full((len(ctx), max(max(used), 1)), -1, dtype=torch.int32)
    at, kv = 0, []
    for b, c in enumerate(ctx):
        table[b, :used[b]] = order[at:at + used[b]]
        at += used[b]
        k, v = normal(g, c, hk, d) * spread, normal(g, c, hk, d) + 0.3
        if c:
            t = torch.arange(c)
            slots = (table[b].long()[t // page] * page + t % page).cuda()
            mbw.kv4_append(cache, k, v, slots)
        n, s, m = ref.quantize(k, group)
        kv.append((n * s + m, ref.quantize(v, group)))
    return cache, table.cuda(), kv, g


def check(out, lse, want, want_lse, mass, fp32=False):
    # each weight p s is rounded to fp16 (2^-11), scores carry some 2^-12 from fp32 sums of up to a few hundred, the
    # result is rounded to bf16 (2^-8)
    tol = mass * 2.0 ** -10 + (0 if fp32 else want.abs() * 2.0 ** -8) + 1e-6
    err = (ref.f64(out) - want).abs()
    assert (err <= tol).all(), (float(err.max()), float((err / tol).max()))
    if lse is not None:
        got = ref.f64(lse)
        none = want_lse == -float("inf")
        assert (got[none] == -float("inf")).all() and (got[~none] - want_lse[~none]).abs().le(2.0 ** -11).all()


CASES = [
    # ctx, queries per request, hq, hk, d, group, page, window
    ([1], [1], 28, 4, 128, 64, 16, 0),
    ([1024], [1], 28, 4, 128, 64, 16, 0),
    ([5, 0, 16, 17, 1, 15, 33], [1] * 7, 32, 4, 64, 32, 16, 0),
    ([100, 63, 64, 65], [1] * 4, 8, 8, 128, 32, 32, 0),
    ([31, 300], [1, 1], 16, 1, 256, 64, 64, 0),
    ([2000], [1], 40, 1, 128, 64, 48, 0),
    ([77, 200, 513], [3, 5, 1], 28, 4, 128, 64, 64, 0),
    ([40, 9, 128, 1], [40, 2, 0, 1], 8, 2, 64, 64, 16, 0),
    ([3, 12], [5, 12], 4, 4, 256, 32, 16, 0),
    ([90, 700], [70, 33], 32, 8, 128, 64, 32, 20),
    ([500, 30, 1], [1, 1, 1], 28, 4, 128, 32, 128, 64),
    ([600], [1], 28, 4, 128, 64, 16, 1),
    ([257], [4], 24, 2, 256, 64, 16, 100),
    ([1, 2, 3, 4, 5, 6, 7, 8] * 9, [1] * 72, 4, 2, 128, 64, 16, 0),
    ([4100, 50], [1, 1], 16, 2, 64, 32, 1024, 0),
]


@pytest.mark.parametrize("i", range(len(CASES)))
@pytest.mark.parametrize("space", ["full", "none", "short"])
def test_attention(i, space):
    ctx, nq, hq, hk, d, group, page, window = CASES[i]
    cache, table, kv, g = filled(i, ctx, page, hk, d, group)
    starts = [0]
    for n in nq:
        starts.append(starts[-1] + n)
    wide = normal(g, starts[-1], hq + 3, d)
    q = wide[:, :hq]
    ws = mbw.kv4_attention_workspace(d)
    ws = {"full": ws, "none": None, "short": ws[:ws.numel() // 37 // 16 * 16]}[space]
    want = ref.attention(q, kv, ctx, starts, d ** -0.5, window)
    c = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    kw = {"window": window, "workspace": ws, "return_lse": True}
    s = torch.tensor(starts, dtype=torch.int32, device="cuda")
    out, lse = mbw.kv4_attention(cache, q, table, c, s, **kw)
    check(out, lse, want[0], want[1], want[2])
    again, _ = mbw.kv4_attention(cache, q, table, c, s, **kw)
    assert torch.equal(out, again)  # bitwise, run after run
    if len(set(nq)) == 1:
        uniform, _ = mbw.kv4_attention(cache, q, table, c, **kw)
        assert torch.equal(out, uniform)
    with mbw.output_fp32():
        o32, _ = mbw.kv4_attention(cache, q, table, c, s, **kw)
    assert o32.dtype == torch.float32
    check(o32, None, want[0], want[1], want[2], fp32=True)


def test_attention_scores_of_any_size():
    """A context whose best key grows from token to token, and one key far above all: the running maximum moves."""
    ctx, hq, hk, d = [400, 400], 8, 2, 128
    cache, table, kv, g = filled(50, ctx, 16, hk, d, 64, spread=4.0)
    q = normal(g, 2, hq, d) * 6
    want = ref.attention(q, kv, ctx, [0, 1, 2], 1.0)
    out, lse = mbw.kv4_attention(cache, q, table, torch.tensor(ctx, dtype=torch.int32, device="cuda"), scale=1.0,
                                 return_lse=True, workspace=mbw.kv4_attention_workspace(d))
    # scores of several hundred: fp32 sums are off by up to 2^-24 * 128 * the sum of their terms' sizes
    err = (ref.f64(out) - want[0]).abs()
    assert (err <= want[2] * 2.0 ** -7 + want[0].abs() * 2.0 ** -8 + 1e-6).all()
    assert ((ref.f64(lse) - want[1]).abs() <= want[1].abs() * 2.0 ** -16).all()


def test_attention_nan_that_a_query_sees_is_not_lost():
    ctx, hq, hk, d = [70], 4, 2, 64
    cache, table, _, g = filled(51, ctx, 16, hk, d, 32)
    bad = torch.zeros(1, hk, d, device="cuda").bfloat16()
    bad[0, 1, 3] = float("nan")
    slot = (table[0, 2].long() * 16 + 7).view(1)
    mbw.kv4_append(cache, torch.zeros_like(bad), bad, slot)
    c = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    out = mbw.kv4_attention(cache, normal(g, 1, hq, d), table, c)
    assert out[0, 2:, :32].isnan().all() and not out[0, 2:, 32:].isnan().any() and not out[0, :2].isnan().any()
    # behind a window that ends before it, it does not enter
    out = mbw.kv4_attention(cache, normal(g, 1, hq, d), table, c, window=70 - 40)
    assert not out.isnan().any()


def test_attention_cache_past_four_gigabytes():
    d, hk, page = 256, 8, 64
    num = (1 << 32) // mbw.kv4_page_bytes(page, hk, d, 64) + 40
    ctx = [200, 64, 500]
    cache, table, kv, g = filled(52, ctx, page, hk, d, 64, num_pages=num)
    assert int(table.max()) * cache.pages.shape[1] > 1 << 32
    q = normal(g, 3, 16, d)
    want = ref.attention(q, kv, ctx, [0, 1, 2, 3], d ** -0.5)
    out, lse = mbw.kv4_attention(cache, q, table, torch.tensor(ctx, dtype=torch.int32, device="cuda"), return_lse=True,
                                 workspace=mbw.kv4_attention_workspace(d))
    check(out, lse, *want)


def test_attention_long_context_is_split_and_joined():
    ctx, hq, hk, d = [30000, 70], 8, 2, 128
    cache, table, kv, g = filled(53, ctx, 64, hk, d, 64)
    q = normal(g, 2, hq, d)
    want = ref.attention(q, kv, ctx, [0, 1, 2], d ** -0.5)
    c = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    ws = mbw.kv4_attention_workspace(d)
    for w in (ws, ws[:200000], None, ws):
        out, lse = mbw.kv4_attention(cache, q, table, c, return_lse=True, workspace=w)
        check(out, lse, *want)


def test_attention_padding_requests_and_queries():
    """Lengths of zero or below, requests without queries, queries behind the last request's: zeros, nothing read."""
    ctx, hq, hk, d = [50, 0, 20], 4, 2, 128
    cache, table, kv, g = filled(54, ctx, 16, hk, d, 64)
    q = normal(g, 3, hq, d)
    c = torch.tensor([50, -3, 20], dtype=torch.int32, device="cuda")
    want = ref.attention(q, kv, ctx, [0, 1, 2, 3], d ** -0.5)
    out, lse = mbw.kv4_attention(cache, q, table, c, return_lse=True, workspace=mbw.kv4_attention_workspace(d))
    check(out, lse, *want)
    assert out[1].eq(0).all()
    empty = mbw.kv4_attention(cache, q[:0], table, c)
    assert empty.shape == (0, hq, d)


def test_attention_page_or_length_out_of_range_is_reported():
    ctx, hq, hk, d = [50, 30], 4, 2, 128
    cache, table, kv, g = filled(55, ctx, 16, hk, d, 64)
    q = normal(g, 2, hq, d)
    c = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    want = ref.attention(q, kv, ctx, [0, 1, 2], d ** -0.5)
    for bad in (-7, 1 << 30):
        t = table.clone()
        t[1, 0] = bad
        out = mbw.kv4_attention(cache, q, t, c, workspace=mbw.kv4_attention_workspace(d))
        with pytest.raises(mbw.MbwError) as e:
            mbw.check_device_error()
        assert e.value.status == 8
        check(out[:1], None, want[0][:1], want[1][:1], want[2][:1])  # the other request is as it was
    mbw.kv4_attention(cache, q, table, torch.tensor([50, 1000], dtype=torch.int32, device="cuda"))
    with pytest.raises(mbw.MbwError):
        mbw.check_device_error()
    mbw.check_device_error()


def test_on_another_stream_and_in_a_graph():
    """Append and attention captured as one graph, replayed with other inputs in the same buffers."""
    hq, hk, d, page = 28, 4, 128, 16
    ctx0 = 90
    cache, table, _, g = filled(56, [ctx0 + 4], page, hk, d, 64)
    qkv = normal(g, 1, hq + 2 * hk, d)
    rope = mbw.rope_table(500, d)
    pos = torch.tensor([ctx0], dtype=torch.int32, device="cuda")
    slot = (table[0, ctx0 // page].long() * page + ctx0 % page).view(1)
    c = torch.tensor([ctx0 + 1], dtype=torch.int32, device="cuda")
    ws = mbw.kv4_attention_workspace(d)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        q = mbw.kv4_append(cache, qkv[:, hq:hq + hk], qkv[:, hq + hk:], slot, q=qkv[:, :hq], positions=pos, cos_sin=rope)
        return mbw.kv4_attention(cache, q, table, c, workspace=ws)

    with torch.cuda.stream(side):
        step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            out = step()
    for seed in range(3):
        qkv.copy_(normal(gen(seed), 1, hq + 2 * hk, d))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, step())


def test_injected_launch_failures():
    cache = new_cache(2, 16, 1, 64, 32)
    x = normal(gen(1), 1, 1, 64)
    s = torch.zeros(1, dtype=torch.int64, device="cuda")
    t, c = torch.zeros(1, 1, dtype=torch.int32, device="cuda"), torch.ones(1, dtype=torch.int32, device="cuda")
    for call in (lambda: mbw.kv4_append(cache, x, x, s), lambda: mbw.kv4_gather(cache, s),
                 lambda: mbw.kv4_attention(cache, x, t, c), lambda: mbw.token_logprobs(x[0])):
        n = mbw.launch_count()
        mbw.inject_launch_failures(1)
        with pytest.raises(mbw.MbwError) as e:
            call()
        assert e.value.status == 6 and mbw.launch_count() == n
        call()
        assert mbw.launch_count() > n
    assert B.lib().mbw_kv4_page_bytes(16, 1, 64, 32) == mbw.kv4_page_bytes(16, 1, 64, 32)
