"""The decode example with 8-bit floating point products and with prompts that
share their beginning: the operators run together, eagerly and as one CUDA graph."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - the marker keeps these off CPU runs
    pytest.skip("needs a GPU", allow_module_level=True)

import memory_bound_weight_gb300 as mbw  # noqa: E402
from memory_bound_weight_gb300.decode import Decoder, Shape  # noqa: E402
from test_fp8_gpu import check, exact, half_step, plain_rows  # noqa: E402

SMALL = Shape(hidden=512, heads=14, kv_heads=2, dim=64, mlp=1024, vocab=5003, layers=2, rope_base=1e4)
FRONT = [(7 * i * i + 3 * i + 11) % 5003 for i in range(100)]
PROMPTS = [FRONT + [3, 1, 4, 1, 5, 9, 2, 6, 5, 3, 5, 8, 9, 7, 9, 3, 2], FRONT + [2, 7, 1], FRONT + [8] * 40]


def check_product(d, w, x, norm, up, residual, got):
    """A product of the run against its definition on the inputs that it had (tests/test_fp8_gpu.py's bounds)."""
    rows = x
    if norm is not None:
        r = (1 / (x.double().pow(2).mean(-1, keepdim=True) + 1e-6).sqrt()).float()
        rows = (x.float() * r * norm.float()).bfloat16()
    q, sc = plain_rows(rows)
    y, mass, eps = exact(q, sc, *w)
    tol = mass * eps
    if up is not None:
        u, mass_u, _ = exact(q, sc, *up)
        act = y * torch.sigmoid(y)
        tol = 1.1 * tol * u.abs() + act.abs() * mass_u * eps + 1.1 * mass * mass_u * eps * eps + (act * u).abs() * 2.0 ** -20
        y = act * u
    if residual is not None:
        y = y + residual.double()
        tol = tol + y.abs() * 2.0 ** -24
    check(got, y, tol + half_step(y))


def check_attention(d, cache, q, q_starts, got):
    """Attention behind shared pages against that over each request's own table. Values are some units in size; a weight is off
    by 2^-11 and what its score is, some 2^-8 here, either way, which acts on the distance of a value from the result; outputs
    are rounded by 2^-8 each."""
    want = mbw.kv4_attention(cache, q, d.table, d.ctx, q_starts).float()
    assert ((got.float() - want).abs() <= 2.0 ** -6 + want.abs() * 2.0 ** -7).all()


@pytest.mark.parametrize("weights,share", [("fp8", False), ("bf16", True), ("fp8", True)])
def test_every_operator_of_a_run_follows_its_definition(weights, share, monkeypatch):
    d = Decoder(SMALL, requests=3, max_tokens=200, weights=weights)
    product, attend, ran = d.product, d.attend, []

    def checked_product(w, x, norm=None, up=None, residual=None):
        before = None if residual is None else residual.clone()
        out = product(w, x, norm=norm, up=up, residual=residual)
        if weights == "fp8":
            check_product(d, w, x, norm, up, before, out)
        ran.append(len(x))
        return out

    def checked_attend(cache, q, q_starts):
        out = attend(cache, q, q_starts)
        if d.shared:
            check_attention(d, cache, q, q_starts, out)
        return out

    monkeypatch.setattr(d, "product", checked_product)
    monkeypatch.setattr(d, "attend", checked_attend)
    r = d.prompt(PROMPTS, share=share)
    assert d.shared == (96 if share else 0) and d.ctx.tolist() == [len(p) for p in PROMPTS]
    n = [len(p) for p in PROMPTS]
    chunks = [96, sum(n) - 3 * 96] if share else [sum(n)]
    assert ran == [t for t in chunks for _ in range(2 * 4)] + [3]
    for _ in range(4):
        r = d.step(top_k=2)
    assert all(x.isfinite().all() for x in (r.entropy, r.top_logprobs)) and len(ran) == 4 * 2 * (len(chunks) + 4) + 5


@pytest.mark.parametrize("weights,share", [("fp8", False), ("bf16", True), ("fp8", True)])
def test_graphs_follow_steps(weights, share):
    a, b = (Decoder(SMALL, requests=3, max_tokens=200, weights=weights) for _ in range(2))
    for d in (a, b):
        d.prompt(PROMPTS, share=share)
    replay, out = b.graph(top_k=3)
    for _ in range(30):  # over the ends of pages
        r = a.step(top_k=3)
        replay()
        torch.cuda.synchronize()
        for u, v in zip(r, out):
            assert u is None and v is None or torch.equal(u, v)
    assert a.ctx.tolist() == [len(p) + 30 for p in PROMPTS] and torch.equal(a.ids, b.ids)


def test_shared_pages_are_held_once_and_left_by_the_next_prompts():
    d = Decoder(SMALL, requests=3, max_tokens=200)
    d.prompt(PROMPTS, share=True)
    assert (d.table[:, :6] == d.table[:1, :6]).all() and not (d.table[1:, 6] == d.table[0, 6]).any()
    d.prompt([[3, 1, 4], [2, 7, 1, 8], [5]], share=True)  # nothing in common
    assert d.shared == 0 and torch.equal(d.table, d.own_table)
    d.prompt([FRONT[:33]] * 3, share=True)  # the same prompt: two pages, and the last token each request's own
    assert d.shared == 32
    one = Decoder(SMALL, requests=1, max_tokens=200)
    r = one.prompt([FRONT[:33]])
    assert torch.equal(d.ids, r.top_ids[:, 0].expand(3).long())


def test_a_step_of_many_requests_attends_to_the_shared_pages_once():
    """So many requests that the shared pages have their kernel; then a step's log probabilities are those of requests in
    their own pages but for what roundings move (as above)."""
    shape = Shape(hidden=512, heads=32, kv_heads=8, dim=128, mlp=512, vocab=1009, layers=1, rope_base=1e4)
    front = [(5 * i * i + i) % 1009 for i in range(2500)]
    prompts = [front + [i % 1009, 3, (7 * i) % 1009][:1 + i % 3] for i in range(64)]
    a, b = (Decoder(shape, requests=64, max_tokens=2600) for _ in range(2))
    a.prompt(prompts, share=True)
    b.prompt(prompts)
    assert a.shared == 2496
    a.ids.copy_(torch.arange(64, device="cuda"))
    b.ids.copy_(a.ids)
    n = mbw.launch_count()
    x = a.step()
    m = mbw.launch_count()
    y = b.step()
    assert m - n == mbw.launch_count() - m + 1
    # One layer whose attention is off by 2^-6 at most (above) where its outputs are bf16 rows of size 1: the logits of a
    # normed row move by as much of their spread, about 1, and the entropy of 1009 tokens by less.
    assert (x.entropy - y.entropy).abs().max() < 2.0 ** -4
