"""The compiled marshalling of the cache and token calls: it takes the ordinary calls, gives what the Python functions give,
and leaves everything else to them, their refusals included."""
import pytest
import torch

import memory_bound_weight_gb300 as mbw
from memory_bound_weight_gb300 import _binding as B
from test_kv4_gpu import gen, new_cache, normal

pytestmark = pytest.mark.gpu


def python_only(monkeypatch, f):
    with monkeypatch.context() as m:
        m.setattr(B, "_fast", False)
        return f()


def setup(T=5, hq=8, hk=2, d=128):
    g = gen(80)
    wide = normal(g, T, hq + 2 * hk, d)
    cache = new_cache(4, 16, hk, d, 64)
    slots = torch.arange(T, device="cuda") + 20
    pos = torch.arange(T, device="cuda", dtype=torch.int32) * 3
    return cache, wide[:, :hq], wide[:, hq:hq + hk], wide[:, hq + hk:], slots, pos, mbw.rope_table(64, d)


def test_it_is_there_and_gives_the_same(monkeypatch):
    cache, q, k, v, slots, pos, cs = setup()
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    ctx = torch.tensor([9], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0, 5], dtype=torch.int32, device="cuda")
    ws, lws = mbw.kv4_attention_workspace(128), mbw.token_logprobs_workspace()
    logits = normal(gen(81), 3, 4000)
    target = torch.tensor([1, 2, 3999], dtype=torch.int32, device="cuda")

    def calls():
        out = [mbw.kv4_append(cache, k, v, slots, q=q, positions=pos, cos_sin=cs),
               mbw.kv4_append(cache, k, v, slots, q=q, positions=pos, cos_sin=cs, interleaved=True, q_out=torch.zeros_like(q)),
               *mbw.kv4_gather(cache, slots), mbw.kv4_attention(cache, q, table, ctx, starts, workspace=ws)]
        out += mbw.kv4_attention(cache, q, table, ctx, starts, scale=0.1, window=3, return_lse=True)
        out += mbw.token_logprobs(logits, target, top_k=4, workspace=lws)
        out += mbw.token_logprobs(logits, top_k=2)[2:]
        assert mbw.kv4_append(cache, k, v, slots) is None
        r = mbw.token_logprobs(logits)
        assert isinstance(r, B.TokenLogprobs) and r.logprob is None and r.top_ids.shape == (3, 0)
        return out

    fast = calls()
    assert B._fast and B._fast.kv4_gather(cache._addr, cache.pages, slots) is not None
    slow = python_only(monkeypatch, calls)
    for x, y in zip(fast, slow):
        assert x.dtype == y.dtype and x.shape == y.shape and torch.equal(x.nan_to_num(), y.nan_to_num())


@pytest.mark.parametrize("wrong", ["dtype", "shape", "device", "tokens", "half", "kind"])
def test_what_is_wrong_is_refused_in_the_same_words(monkeypatch, wrong):
    cache, q, k, v, slots, pos, cs = setup()

    def call():
        if wrong == "dtype":
            return mbw.kv4_append(cache, k, v.float(), slots)
        if wrong == "shape":
            return mbw.kv4_append(cache, k, v[:, :1], slots)
        if wrong == "device":
            return mbw.kv4_gather(cache, slots.cpu())
        if wrong == "tokens":
            return mbw.kv4_append(cache, k, v, slots[:-1])
        if wrong == "half":
            return mbw.kv4_append(cache, k, v, slots, q=q, positions=pos)
        return mbw.token_logprobs(torch.zeros(2, 8, dtype=torch.float16, device="cuda"))

    said = []
    for f in (call, lambda: python_only(monkeypatch, call)):
        with pytest.raises((TypeError, ValueError)) as e:
            f()
        said.append((e.type, str(e.value)))
    assert said[0] == said[1]


def test_the_librarys_refusals_and_failures_raise():
    cache, q, k, v, slots, pos, cs = setup()
    with pytest.raises(mbw.MbwError):  # rotary dimension that is no multiple of 16
        mbw.kv4_append(cache, k, v, slots, q=q, positions=pos, cos_sin=torch.zeros(64, 24, device="cuda"))
    mbw.inject_launch_failures(1)
    with pytest.raises(mbw.MbwError):
        mbw.kv4_gather(cache, slots)
    mbw.kv4_gather(cache, slots)


def test_whole_numbers_and_other_workspaces_are_left_to_python():
    cache, q, k, v, slots, pos, cs = setup()
    mbw.kv4_append(cache, k, v, slots, q=q, positions=pos, cos_sin=cs)
    table = torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
    ctx = torch.tensor([9], dtype=torch.int32, device="cuda")
    a = mbw.kv4_attention(cache, q, table, ctx, scale=1)
    b = mbw.kv4_attention(cache, q, table, ctx, scale=1.0)
    c = mbw.kv4_attention(cache, torch.nn.Parameter(q.clone(), requires_grad=False), table, ctx, scale=1.0)
    assert torch.equal(a.nan_to_num(), b.nan_to_num()) and torch.equal(a.nan_to_num(), c.nan_to_num())
    assert not a.requires_grad and not c.requires_grad
