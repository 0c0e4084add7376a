"""The decode example's shared beginnings, on the host. A captured step is refused behind prompts that share fewer tokens than
those it was captured for: their length is part of what was captured, and the pages it names would be another request's. Where
the beginning's own pass fails, no request is left in another's pages."""
import pytest

torch = pytest.importorskip("torch")

from memory_bound_weight_gb300.decode import Decoder, Shape  # noqa: E402

SMALL = Shape(hidden=512, heads=14, kv_heads=2, dim=64, mlp=1024, vocab=50, layers=2, rope_base=1e4)


@pytest.fixture
def decoder(monkeypatch):
    """A decoder of 3 requests whose layers, on no GPU, do nothing."""
    d = object.__new__(Decoder)
    d.shape, d.requests, d.max_tokens, d.page_size, d.longest = SMALL, 3, 100, 16, 0
    d.ctx, d.ids = torch.zeros(3, dtype=torch.int32), torch.zeros(3, dtype=torch.int64)
    d.own_table = torch.arange(21, dtype=torch.int32).view(3, 7)
    d.table = d.own_table.clone()
    monkeypatch.setattr(d, "forward", lambda ids, *a: None, raising=False)
    monkeypatch.setattr(d, "choose", lambda logits, top_k=1: top_k, raising=False)
    return d


def prompts(shared):
    return [[7] * shared + [i + 1] for i in range(3)]


def test_a_step_captured_behind_a_shared_beginning_needs_it(decoder):
    decoder.prompt(prompts(48), share=True)
    assert decoder.shared == 48
    replayed = []
    replay = decoder.counted(lambda: replayed.append(decoder.shared))
    replay()
    for shared, share in ((32, True), (0, True), (48, False)):
        decoder.prompt(prompts(shared), share=share)
        assert decoder.shared == (shared if share else 0)
        longest = decoder.longest
        with pytest.raises(ValueError, match="share"):
            replay()
        assert decoder.longest == longest  # nothing was counted
    assert replayed == [48]
    for shared in (48, 64):  # as many, and more, which are then as good as each request's own
        decoder.prompt(prompts(shared), share=True)
        replay()
    assert replayed == [48, 48, 64]


def test_a_step_captured_without_one_follows_any_prompt(decoder):
    decoder.prompt(prompts(5), share=True)  # no whole page
    assert decoder.shared == 0
    replayed = []
    replay = decoder.counted(lambda: replayed.append(decoder.shared))
    for shared, share in ((64, True), (16, True), (64, False)):
        decoder.prompt(prompts(shared), share=share)
        replay()
    assert replayed == [64, 16, 0]


def test_a_beginning_that_fails_leaves_each_request_in_its_own_pages(decoder, monkeypatch):
    def fails(*a):
        raise RuntimeError("no memory")

    with monkeypatch.context() as m:
        m.setattr(decoder, "forward", fails, raising=False)
        with pytest.raises(RuntimeError, match="no memory"):
            decoder.prompt(prompts(48), share=True)
    assert decoder.shared == 0 and torch.equal(decoder.table, decoder.own_table)
    decoder.prompt(prompts(48))
    assert torch.equal(decoder.table, decoder.own_table)
    decoder.prompt(prompts(48), share=True)
    assert decoder.shared == 48 and (decoder.table[:, :3] == decoder.table[:1, :3]).all()
