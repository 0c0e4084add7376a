"""The decode example: its products, cache, attention and log probabilities run
together, eagerly and as one CUDA graph."""
import pytest

import kv4_ref as ref

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():  # pragma: no cover - the marker keeps these off CPU runs
    pytest.skip("needs a GPU", allow_module_level=True)

import memory_bound_weight_gb300 as mbw  # noqa: E402
from memory_bound_weight_gb300.decode import Decoder, Shape  # noqa: E402

SMALL = Shape(hidden=512, heads=14, kv_heads=2, dim=64, mlp=1024, vocab=5003, layers=2, rope_base=1e4)
PROMPTS = [[3, 1, 4, 1, 5, 9, 2, 6, 5, 3, 5, 8, 9, 7, 9, 3, 2], [2, 7, 1], [8] * 40]


def norm(x, w, eps=1e-6):
    return (x * w / (x.pow(2).mean(-1, keepdim=True) + eps).sqrt()).bfloat16().double()


def plain_logits(d, prompts):
    """The model over whole prompts in 64 bits, with a rounding to bf16 where the step has a bf16 tensor, and keys and
    values as the cache holds them."""
    out, s = [], d.shape
    for p in prompts:
        x = d.embedding[torch.tensor(p, device="cuda")].cpu().double()
        pos = torch.arange(len(p))
        for w in d.layers:
            w = {k: v.cpu().double() for k, v in w.items()}
            qkv = (norm(x, w["norm1"]) @ w["qkv"].T).bfloat16().view(len(p), -1, s.dim)
            q, k, v = qkv.split((s.heads, s.kv_heads, s.kv_heads), 1)
            q, k = (ref.rotate(t, d.cos_sin, pos, False).float().bfloat16() for t in (q, k))
            n, sc, m = ref.quantize(k, 64)
            a, _, _ = ref.attention(q, [(n * sc + m, ref.quantize(v, 64))], [len(p)], [0, len(p)], s.dim ** -0.5)
            x = (a.bfloat16().double().view(len(p), -1) @ w["o"].T + x).bfloat16().double()
            h = norm(x, w["norm2"])
            g = torch.nn.functional.silu(h @ w["gate"].T) * (h @ w["up"].T)
            x = (g.bfloat16().double() @ w["down"].T + x).bfloat16().double()
        out.append((norm(x[-1:], d.norm.cpu().double()) @ d.head.cpu().double().T)[0])
    return torch.stack(out)


def test_prompt_follows_the_formulas():
    d = Decoder(SMALL, requests=3, max_tokens=100)
    r = d.prompt(PROMPTS)
    want = torch.log_softmax(plain_logits(d, PROMPTS), -1)
    # Logits of about unit size. Each layer rounds five tensors to bf16 (2^-9 on average), and a key or value that falls
    # on the other side of a border moves a code by one step of 15, in a mean over the context: some 2^-6 of the
    # logits' spread over two layers; held to 2^-4.
    got = r.top_logprobs[:, 0].cpu().double()
    there = want.gather(1, r.top_ids.cpu().long())[:, 0]
    assert (got - there).abs().max() < 2.0 ** -4
    assert (there >= want.max(-1).values - 2.0 ** -3).all()  # the chosen token is the best but for near ties
    ent = -(want.exp() * want).sum(-1)
    assert (r.entropy.cpu().double() - ent).abs().max() < 2.0 ** -4


def test_steps_follow_the_prompt_and_graphs_follow_steps():
    a, b = Decoder(SMALL, requests=3, max_tokens=100), Decoder(SMALL, requests=3, max_tokens=100)
    for d in (a, b):
        d.prompt(PROMPTS)
    replay, out = b.graph(top_k=3)
    assert torch.equal(a.ids, b.ids) and torch.equal(a.ctx, b.ctx)
    for _ in range(30):  # over the ends of pages
        r = a.step(top_k=3)
        replay()
        torch.cuda.synchronize()
        for u, v in zip(r, out):
            assert u is None and v is None or torch.equal(u, v)
    assert a.ctx.tolist() == [len(p) + 30 for p in PROMPTS] and torch.equal(a.ids, b.ids)
    # the tokens that a's last step wrote are in the cache: read back, they are the formula's values of some bf16 row
    last = a.ctx.long() - 1
    slots = a.table[torch.arange(3, device="cuda"), last // 16].long() * 16 + last % 16
    for x, y in zip(a.caches, b.caches):
        for u, v in zip(mbw.kv4_gather(x, slots), mbw.kv4_gather(y, slots)):
            assert torch.equal(u, v) and u.isfinite().all() and u.abs().max() > 0
