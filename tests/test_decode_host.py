"""The decode example refuses, on the host and before anything runs, what would index past its tables on the device."""
import pytest

torch = pytest.importorskip("torch")

from memory_bound_weight_gb300.decode import Decoder, Shape  # noqa: E402

SMALL = Shape(hidden=512, heads=14, kv_heads=2, dim=64, mlp=1024, vocab=50, layers=2, rope_base=1e4)


@pytest.fixture
def decoder(monkeypatch):
    """A decoder of 2 requests of up to 20 tokens whose layers, on no GPU, count their calls."""
    d = object.__new__(Decoder)
    d.shape, d.requests, d.max_tokens, d.page_size, d.longest = SMALL, 2, 20, 16, 0
    d.ctx, d.ids, d.ran = torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int64), []
    monkeypatch.setattr(d, "forward", lambda ids, *a: d.ran.append(len(ids)), raising=False)
    monkeypatch.setattr(d, "choose", lambda logits, top_k=1: top_k, raising=False)
    return d


def test_steps_end_at_the_tables_end(decoder):
    decoder.prompt([[1, 2, 3], [4] * 17])
    for _ in range(3):
        decoder.step()
    assert decoder.ran == [20, 2, 2, 2] and decoder.ctx.tolist() == [6, 20]
    for _ in range(2):
        with pytest.raises(ValueError, match="max_tokens"):
            decoder.step()
    assert len(decoder.ran) == 4 and decoder.ctx.tolist() == [6, 20]
    decoder.prompt([[1], [2]])  # from the start again
    decoder.step()
    assert len(decoder.ran) == 6


@pytest.mark.parametrize("prompts,words", [
    ([[1] * 21, [1]], "max_tokens"), ([[1]], "2 prompts"), ([[1], [2], [3]], "2 prompts"), ([[1], []], "empty"),
    ([[1], [50]], "id"), ([[-1], [3]], "id"),
])
def test_prompts_that_do_not_fit_are_refused(decoder, prompts, words):
    with pytest.raises(ValueError, match=words):
        decoder.prompt(prompts)
    assert decoder.ran == [] and decoder.ctx.tolist() == [0, 0]


def test_replays_end_at_the_tables_end(decoder):
    decoder.prompt([[1], [4] * 18])
    replayed = []
    replay = decoder.counted(lambda: replayed.append(1))
    replay()
    decoder.step()
    with pytest.raises(ValueError, match="max_tokens"):
        replay()
    assert replayed == [1]


def test_no_graph_is_captured_behind_the_last_place(decoder):
    decoder.prompt([[1], [4] * 20])
    with pytest.raises(ValueError, match="max_tokens"):
        decoder.graph()
    assert decoder.ran == [21]
