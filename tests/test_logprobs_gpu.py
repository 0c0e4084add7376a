"""Log probabilities of tokens on the GPU against the definition in 64 bits."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - the marker keeps these off CPU runs
    pytest.skip("needs a GPU", allow_module_level=True)

import memory_bound_weight_gb300 as mbw  # noqa: E402

INF = float("inf")


def reference(x, t, k, scale):
    """(logprob, rank, entropy, ids, logprobs of ids) in 64 bits, ties to the lower id."""
    x = x.detach().double()
    y = torch.log_softmax(x * scale, -1)
    dead = (x == -INF).all(-1)
    y[dead] = -INF
    ent = -torch.where(y > -INF, y.exp() * y, 0.0).sum(-1)
    order = torch.sort(x + 0.0, dim=-1, descending=True, stable=True).indices
    ids = order[:, :k].clone()
    top = y.gather(1, ids)
    if ids.shape[1] < k:  # fewer tokens than asked for
        more = k - ids.shape[1]
        ids = torch.cat((ids, ids.new_full((len(ids), more), -1)), 1)
        top = torch.cat((top, top.new_full((len(top), more), -INF)), 1)
    ids[top == -INF] = -1
    lp = rank = None
    if t is not None:
        none = t < 0
        tt = t.long().clamp(min=0)[:, None]
        lp = torch.where(none, 0.0, y.gather(1, tt)[:, 0])
        place = torch.empty_like(order).scatter_(1, order, torch.arange(x.shape[1], device=x.device).expand_as(order))
        rank = torch.where(none, 0, place.gather(1, tt)[:, 0] + 1)
    return lp, rank, ent, ids, top


def near(got, want):
    """Differences and logarithms of relative error 2^-22, sums of positive terms in fp32 of relative error 2^-20, which
    moves their logarithm by as much."""
    got = got.double()
    fine = want.isfinite()
    assert torch.equal(got[~fine], want[~fine])
    got, want = got[fine], want[fine]
    assert ((got - want).abs() <= 2.0 ** -20 + want.abs() * 2.0 ** -21).all(), float((got - want).abs().max())


def compare(x, t, k, scale=1.0, workspace=None):
    r = mbw.token_logprobs(x, t, top_k=k, scale=scale, workspace=workspace)
    lp, rank, ent, ids, top = reference(x, t, k, scale)
    near(r.top_logprobs, top)
    assert torch.equal(r.top_ids.long(), ids)
    near(r.entropy, ent)
    if t is None:
        assert r.logprob is None and r.rank is None
    else:
        near(r.logprob, lp)
        assert torch.equal(r.rank.long(), rank)
    return r


@pytest.mark.parametrize("M,V,k,dtype,scale", [
    (1, 1, 1, "bf16", 1.0), (3, 2, 5, "fp32", 1.0), (2, 7, 32, "bf16", 2.0), (5, 8, 0, "bf16", 1.0),
    (4, 255, 20, "fp32", 0.5), (1, 1000, 1, "bf16", 1.0), (33, 1001, 32, "bf16", 1.0), (7, 32000, 8, "fp32", 1.3),
    (1, 152064, 20, "bf16", 1.0), (2, 151936, 32, "fp32", 1.0), (300, 5003, 5, "bf16", 0.7),
    (1000, 2048, 1, "bf16", 1.0), (160, 33001, 20, "bf16", 1.0), (64, 152064, 0, "bf16", 1.0),
])
@pytest.mark.parametrize("space", [True, False])
def test_random_rows(M, V, k, dtype, scale, space):
    g = torch.Generator(device="cuda")
    g.manual_seed(M * V)
    x = torch.randn(M, V, generator=g, device="cuda") * 4
    x = x.bfloat16() if dtype == "bf16" else x
    t = torch.randint(V, (M,), generator=g, device="cuda").to(torch.int32)
    if M > 2:
        t[1] = -1
    ws = mbw.token_logprobs_workspace() if space else None
    a = compare(x, t, k, scale, ws)
    b = mbw.token_logprobs(x, t, top_k=k, scale=scale, workspace=ws)
    for u, v in zip(a, b):
        assert torch.equal(u, v)  # bitwise, run after run


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("offset,pad", [(0, 3), (1, 5), (5, 8)])
def test_rows_that_start_anywhere(dtype, offset, pad):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    M, V = 5, 4099
    x = (torch.randn(M, V + pad + offset, device="cuda") * 3).to(dt)[:, offset:offset + V]
    t = torch.tensor([0, V - 1, 5, 4096, -1], dtype=torch.int32, device="cuda")
    for ws in (None, mbw.token_logprobs_workspace()):
        compare(x, t, 9, workspace=ws)


@pytest.mark.parametrize("V", [64, 40000, 152064])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_ties_masks_and_orders(V, dtype):
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    low = torch.finfo(dt).min
    up = torch.arange(V, device="cuda", dtype=torch.float32) / V * 20
    rows = [torch.zeros(V, device="cuda"), up, up.flip(0), torch.full((V,), -INF, device="cuda"),
            torch.full((V,), low, device="cuda"), (up % 1).round(), torch.full((V,), -INF, device="cuda"),
            torch.full((V,), low, device="cuda"), -up.square() * 100, torch.full((V,), -INF, device="cuda"),
            torch.full((V,), -0.0, device="cuda")]
    rows[6][V // 2] = -3.0  # one token allowed
    rows[7][V // 3], rows[7][V // 3 + 9] = 5.0, 5.0
    rows[9][::7] = low  # only the type's lowest value is left
    rows[10][3::5] = 0.0  # zeros of both signs tie
    x = torch.stack(rows).to(dt)
    for t in (0, V - 1, V // 2):
        tt = torch.full((len(rows),), t, dtype=torch.int32, device="cuda")
        for ws in (None, mbw.token_logprobs_workspace()):
            compare(x, tt, 32, workspace=ws)
    assert mbw.token_logprobs(x[3:4]).entropy.item() == 0.0


def test_a_sure_token_keeps_its_digits():
    """log p of a token that has nearly all the probability, and the entropy, keep relative accuracy."""
    V = 50000
    x = torch.full((3, V), -25.0, device="cuda")
    x[0, 77], x[1, 5], x[2, V - 1] = 3.0, 10.0, 0.0
    t = torch.tensor([77, 5, V - 1], dtype=torch.int32, device="cuda")
    for ws in (None, mbw.token_logprobs_workspace()):
        r = mbw.token_logprobs(x, t, top_k=1, workspace=ws)
        d = x.double()
        gap = d - d.amax(-1, keepdim=True)
        s = torch.where(gap < 0, gap.exp(), 0.0).sum(-1)
        lp = -torch.log1p(s)
        ent = torch.log1p(s) - torch.where(gap < 0, gap.exp() * gap, 0.0).sum(-1) / (1 + s)
        assert ((r.logprob.double() / lp - 1).abs() < 2.0 ** -18).all()
        assert ((r.entropy.double() / ent - 1).abs() < 2.0 ** -18).all()
        assert torch.equal(r.top_logprobs[:, 0], r.logprob)


@pytest.mark.parametrize("bad", [float("nan"), INF])
@pytest.mark.parametrize("place", [0, 17, 39999])
def test_nan_and_infinity_are_not_lost(bad, place):
    x = torch.randn(3, 40000, device="cuda").bfloat16()
    x[1, place] = bad
    t = torch.tensor([3, 4, 5], dtype=torch.int32, device="cuda")
    for ws in (None, mbw.token_logprobs_workspace()):
        r = mbw.token_logprobs(x, t, top_k=3, workspace=ws)
        assert r.logprob[1].isnan() and r.entropy[1].isnan() and r.top_logprobs[1].isnan().all()
        for u in (r.logprob, r.entropy, r.top_logprobs):
            assert u[0].isfinite().all() and u[2].isfinite().all()


def test_target_out_of_range_is_reported():
    x = torch.randn(2, 100, device="cuda")
    r = mbw.token_logprobs(x, torch.tensor([100, 3], dtype=torch.int32, device="cuda"))
    assert r.logprob[0] == 0 and r.rank[0] == 0 and r.rank[1] > 0
    with pytest.raises(mbw.MbwError) as e:
        mbw.check_device_error()
    assert e.value.status == 8
    mbw.check_device_error()


def test_offsets_past_32_bits():
    V, M = 152064, 15000  # 2.28e9 elements
    x = torch.zeros(M, V, dtype=torch.bfloat16, device="cuda")
    x[-1] = torch.randn(V, device="cuda") * 3
    x[-2, 9] = 4.0
    t = torch.full((M,), 9, dtype=torch.int32, device="cuda")
    r = mbw.token_logprobs(x, t, top_k=2, workspace=mbw.token_logprobs_workspace())
    lp, rank, ent, ids, top = reference(x[-2:], t[-2:], 2, 1.0)
    near(r.logprob[-2:], lp)
    near(r.entropy[-2:], ent)
    assert torch.equal(r.top_ids[-2:].long(), ids) and torch.equal(r.rank[-2:].long(), rank)
    assert (r.rank[:-2] == 10).all()


def test_graph_and_other_stream():
    x = torch.randn(4, 32000, device="cuda").bfloat16()
    t = torch.arange(4, dtype=torch.int32, device="cuda")
    ws = mbw.token_logprobs_workspace()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        mbw.token_logprobs(x, t, top_k=5, workspace=ws)
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            r = mbw.token_logprobs(x, t, top_k=5, workspace=ws)
    for _ in range(2):
        x.copy_(torch.randn(4, 32000, device="cuda"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = mbw.token_logprobs(x, t, top_k=5)
        assert torch.equal(r.top_ids, want.top_ids) and torch.equal(r.rank, want.rank)
        lp = reference(x, t, 5, 1.0)[0]
        near(r.logprob, lp)
