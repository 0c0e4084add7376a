"""Measured cases of the operators around the weight-streaming products of a
decode step: the 4-bit paged key/value cache (appending to it with the position
rotation, attention over it) and the log probabilities of tokens.

Each case is one call as a serving engine makes it. ``run`` computes it in its
plain form (elementary torch operations, 32 bits) or, with ``own`` set, through
the package's entry points. ``exact`` is the operators' definition in 64 bits.

The cache holds blocks of 16 tokens of one KV head: 4-bit codes of K and V and,
per token and group of G dimensions, an fp16 scale and an fp16 minimum; a value
is scale * code + minimum.
"""
import math

import torch

own = False

# Head layouts (query heads, KV heads, head dimension) of the package's model
# workloads: Qwen2.5-7B, TinyLlama-1.1B, Qwen3-4B; and a generic wide head.
QWEN25 = {"heads": 28, "kv_heads": 4, "dim": 128}
TINYLLAMA = {"heads": 32, "kv_heads": 4, "dim": 64}
QWEN3 = {"heads": 32, "kv_heads": 8, "dim": 128}
WIDE = {"heads": 16, "kv_heads": 8, "dim": 256}
LAYOUTS = (QWEN25, TINYLLAMA, QWEN3, WIDE)


def _attn(name, layout, batch, lo, hi, q_lo=1, q_hi=1, page=16, group=64, window=0):
    return {"name": name, "op": "attention", **layout, "batch": batch, "ctx_lo": lo, "ctx_hi": hi, "q_lo": q_lo,
            "q_hi": q_hi, "page": page, "group": group, "window": window}


def _append(name, layout, tokens, rotary, interleaved=False, page=16, group=64, start=0):
    return {"name": name, "op": "append", **layout, "tokens": tokens, "rotary": rotary, "interleaved": interleaved,
            "page": page, "group": group, "start": start}


def _logprob(name, rows, vocab, top, dtype="bf16", masked=False, scale=1.0):
    return {"name": name, "op": "logprobs", "rows": rows, "vocab": vocab, "top": top, "dtype": dtype,
            "masked": masked, "scale": scale}


def listed():
    return [
        # one request early in its answer: latency alone
        _attn("attn 1x1 ctx 1024", QWEN25, 1, 1024, 1024),
        # one request with a long document in front of it
        _attn("attn 1x1 ctx 65536", QWEN25, 1, 65536, 65536, page=64),
        # a full batch of requests of mixed age, one token each
        _attn("attn 64x1 ragged 300-16000", QWEN3, 64, 300, 16000, page=32),
        # many short requests of a small model with narrow heads
        _attn("attn 130x1 ragged 17-900 d64", TINYLLAMA, 130, 17, 900, group=32),
        # verification of drafted tokens: a few queries per request
        _attn("attn 12x(2-5) ragged 500-7000", QWEN25, 12, 500, 7000, 2, 5, page=64),
        # a chunk of a prompt behind its cached part, sliding window
        _attn("attn 3x(90-200) window 2048", QWEN3, 3, 1500, 5000, 90, 200, page=32, window=2048),
        # one decode token of one request
        _append("append 1 token", QWEN25, 1, 128),
        # one decode token of each request of a batch, part of the head rotated
        _append("append 61 tokens interleaved", QWEN3, 61, 64, True, page=32, group=32, start=9000),
        # a prompt
        _append("append 8192 tokens", QWEN25, 8192, 128, page=64),
        # the sampled token of one request, with the top alternatives an API returns
        _logprob("logprobs 1x152064 top 20", 1, 152064, 20),
        # constrained decoding of a batch: most tokens masked away
        _logprob("logprobs 50x151936 masked top 8", 50, 151936, 8, "fp32", True, 1.25),
        # scoring the tokens of a prompt
        _logprob("logprobs 2000x152064 top 1", 2000, 152064, 1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("attention", "attention", "append", "logprobs"))
    layout = rng.choice(LAYOUTS)
    page, group = rng.choice((16, 32, 64, 128)), rng.choice((32, 64))
    if op == "attention":
        batch = _log(rng, 1, 200)
        per_token = layout["kv_heads"] * (layout["dim"] + 8 * (layout["dim"] // group))
        hi = _log(rng, 1, min(65536, 500_000_000 // (batch * per_token)))
        lo = rng.randint(max(1, hi // 40), hi)
        most = rng.choice((1, 1, 1, 8, 200))
        most = min(most, lo, max(1, 600 // batch))
        q_hi = rng.randint(1, most)
        q_lo = rng.randint(1, q_hi)
        if q_hi > 8:  # prompt chunks come with shorter contexts than single tokens
            hi = min(hi, max(q_hi, 400_000 // (batch * q_hi)))
            lo = max(q_hi, min(lo, hi))
            hi = max(hi, lo)
        elif q_hi > 1:
            hi = max(q_hi, min(hi, 7_000_000_000 // (batch * q_hi * layout["heads"] * layout["dim"])))
            lo = max(q_hi, min(lo, hi))
        c = _attn("", layout, batch, lo, hi, q_lo, q_hi, page, group, rng.choice((0, 0, 0, rng.randint(1, 4096))))
    elif op == "append":
        c = _append("", layout, _log(rng, 1, 8192 if layout is not WIDE else 4096),
                    rng.choice((layout["dim"], layout["dim"] // 2, 32)), rng.random() < 0.5, page, group,
                    _log(rng, 1, 100_000))
    else:
        vocab = rng.choice((152064, 151936, 32000, _log(rng, 1000, 200_000)))
        dtype = rng.choice(("bf16", "fp32"))
        rows = _log(rng, 1, min(3000, 280_000_000 // vocab // (2 if dtype == "fp32" else 1)))
        c = _logprob("", rows, vocab, rng.choice((0, 1, 5, 20, 32)), dtype, rng.random() < 0.3,
                     rng.choice((1.0, 1.0, 1.5, 0.7)))
    del c["name"]
    return c


# ------------------------------------------------------------------ sizes ----
def _spread(lo, hi, n, phase):
    """n whole numbers between lo and hi, spread evenly over their logarithm in
    a mixed order (multiples of the golden ratio), always with hi among them."""
    out = []
    for i in range(n):
        f = (i * 0.6180339887498949 + phase) % 1.0
        out.append(min(hi, max(lo, int(round(lo * (hi / lo) ** f)))))
    out[n // 2] = hi
    return out


def _lens(c):
    ctx = _spread(c["ctx_lo"], c["ctx_hi"], c["batch"], 0.31)
    nq = _spread(c["q_lo"], c["q_hi"], c["batch"], 0.77)
    return ctx, [min(n, x) for n, x in zip(nq, ctx)]


def _block_bytes(c):
    return 16 * c["dim"] + 128 * (c["dim"] // c["group"])


def work(case):
    c = case
    if c["op"] == "attention":
        ctx, nq = _lens(c)
        w = c["window"]
        keys = [min(x, w + n - 1) if w else x for x, n in zip(ctx, nq)]
        per_token = c["dim"] + 8 * (c["dim"] // c["group"])  # codes, scales and minima of K and V
        rows = sum(nq) * c["heads"]
        pairs = 0
        for x, n in zip(ctx, nq):
            for p in range(x - n, x):
                pairs += min(p + 1, w) if w else p + 1
        return {"bytes": sum(keys) * c["kv_heads"] * per_token + 4 * rows * c["dim"]
                + 4 * sum(-(-x // c["page"]) for x in keys),
                "flops": 4 * pairs * c["heads"] * c["dim"]}
    if c["op"] == "append":
        t, d, hk = c["tokens"], c["dim"], c["kv_heads"]
        read = 2 * t * (c["heads"] + 2 * hk) * d + 4 * t * c["rotary"] + 12 * t
        wrote = 2 * t * c["heads"] * d + t * hk * (d + 8 * (d // c["group"]))
        back = t * hk * (d + 8 * (d // c["group"])) + 2 * t * 2 * hk * d  # the appended values read back
        return {"bytes": read + wrote + back, "flops": 3 * t * (c["heads"] + hk) * c["rotary"] + 8 * t * hk * 2 * d}
    size = 2 if c["dtype"] == "bf16" else 4
    return {"bytes": c["rows"] * (c["vocab"] * size + 16 + 8 * c["top"]), "flops": 6 * c["rows"] * c["vocab"]}


# ----------------------------------------------------------------- inputs ----
def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = "cuda"

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=g, device=dev, dtype=torch.float32) * (hi - lo) + lo

    s = {"case": dict(c)}
    if c["op"] == "attention":
        ctx, nq = _lens(c)
        hk, d, page = c["kv_heads"], c["dim"], c["page"]
        ng, blocks = d // c["group"], page // 16
        used = [-(-x // page) for x in ctx]
        pages = sum(used) + 3
        n = pages * hk * blocks
        # codes of normal values; the order of independent codes does not matter
        pool = torch.empty(n, _block_bytes(c), dtype=torch.uint8, device=dev)
        for i in range(0, n, 1 << 16):
            m = min(n, i + (1 << 16)) - i
            codes = (normal(m, 32 * d) * 3.2 + 7.5).round_().clamp_(0, 15).to(torch.uint8)
            pool[i:i + m, :16 * d] = codes[:, 0::2] | (codes[:, 1::2] << 4)
            scale = uniform(0.15, 0.35, m, 32 * ng)
            low = -7.5 * scale * uniform(0.9, 1.1, m, 32 * ng)
            pool[i:i + m, 16 * d:] = torch.stack((scale, low), 2).half().view(m, -1).view(torch.uint8)
        s["pages"] = pool.view(pages, -1)
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32)
        table = torch.zeros(len(ctx), max(used), dtype=torch.int32)
        order_h, at = order.cpu(), 0
        for b, u in enumerate(used):
            table[b, :u] = order_h[at:at + u]
            at += u
        s["table"] = table.cuda()
        s["ctx"] = torch.tensor(ctx, dtype=torch.int32, device=dev)
        starts = [0]
        for x in nq:
            starts.append(starts[-1] + x)
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
        # the query part of the projections' output: rows of a wider matrix
        wide = (normal(starts[-1], (c["heads"] + 2 * hk) * d) * 2).bfloat16()
        s["q"] = wide[:, :c["heads"] * d].view(starts[-1], c["heads"], d)
        s["workspace"] = torch.zeros(64 << 20, dtype=torch.uint8, device=dev)
    elif c["op"] == "append":
        t, h, hk, d, page = c["tokens"], c["heads"], c["kv_heads"], c["dim"], c["page"]
        wide = normal(t, (h + 2 * hk) * d)
        wide[:, :(h + hk) * d] *= uniform(0.3, 2.5, (h + hk) * d)  # channels of unequal size, as in trained heads
        wide = wide.bfloat16().view(t, h + 2 * hk, d)
        s["q"], s["k"], s["v"] = wide[:, :h], wide[:, h:h + hk], wide[:, h + hk:]
        pages = -(-t // page) + 3
        s["pages"] = torch.zeros(pages, hk * (page // 16) * _block_bytes(c), dtype=torch.uint8, device=dev)
        order = torch.randperm(pages, generator=g, device=dev)[:-(-t // page)]
        at = torch.arange(t, device=dev)
        slots = order[at // page] * page + at % page
        if t > 8:
            slots[torch.randperm(t, generator=g, device=dev)[:max(1, t // 100)]] = -1  # padding tokens
        s["slots"] = slots.to(torch.int64)
        s["positions"] = (c["start"] + at).to(torch.int32)
        r = c["rotary"]
        freq = torch.pow(torch.tensor(1e6, dtype=torch.float64, device=dev),
                         -torch.arange(0, r, 2, dtype=torch.float64, device=dev) / r)
        angle = torch.arange(c["start"] + t, dtype=torch.float64, device=dev)[:, None] * freq
        s["cos_sin"] = torch.cat((angle.cos(), angle.sin()), 1).float()
    else:
        m, v = c["rows"], c["vocab"]
        x = torch.empty(m, v, dtype=torch.bfloat16 if c["dtype"] == "bf16" else torch.float32, device=dev)
        for i in range(0, m, 256):
            x[i:i + 256] = normal(min(m, i + 256) - i, v) * 2.5 - 4
        for _ in range(6):  # a few likely tokens in every row
            x[torch.arange(m, device=dev), torch.randint(v, (m,), generator=g, device=dev)] = \
                (uniform(5, 16, m)).to(x.dtype)
        s["targets"] = torch.randint(v, (m,), generator=g, device=dev).to(torch.int32)
        if c["masked"]:
            keep = torch.rand(m, 1, generator=g, device=dev).square() * 0.2
            for i in range(0, m, 256):
                drop = torch.rand(min(m, i + 256) - i, v, generator=g, device=dev) >= keep[i:i + 256]
                x[i:i + 256].masked_fill_(drop, float("-inf"))
            x[torch.arange(m, device=dev), s["targets"].long()] = 1.0  # the sampled token was allowed
        s["logits"] = x
        s["workspace"] = torch.zeros(8 << 20, dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------------- running ----
def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"attention": _plain_attention, "append": _plain_append, "logprobs": _plain_logprobs}[op](state)


def _own(s, op):
    import memory_bound_weight_gb300 as mbw

    c = s["case"]
    if op == "attention":
        cache = mbw.Kv4Cache(s["pages"], c["kv_heads"], c["dim"], c["page"], c["group"])
        return mbw.kv4_attention(cache, s["q"], s["table"], s["ctx"], s["starts"] if c["q_hi"] > 1 else None,
                                 window=c["window"], workspace=s["workspace"])
    if op == "append":
        cache = mbw.Kv4Cache(s["pages"], c["kv_heads"], c["dim"], c["page"], c["group"])
        q = mbw.kv4_append(cache, s["k"], s["v"], s["slots"], q=s["q"], positions=s["positions"],
                           cos_sin=s["cos_sin"], interleaved=c["interleaved"])
        k, v = mbw.kv4_gather(cache, s["slots"])
        return q, k, v
    r = mbw.token_logprobs(s["logits"], s["targets"], top_k=c["top"], scale=c["scale"], workspace=s["workspace"])
    return {"logprob": r.logprob, "rank": r.rank, "entropy": r.entropy, "top_ids": r.top_ids,
            "top_logprobs": r.top_logprobs}


def _nibbles(x):
    return torch.stack((x & 15, x >> 4), -1).flatten(-2)


def _decode(blocks, d, group):
    """uint8 [..., block bytes] -> K, V fp32 [..., 16, d]."""
    lead, ng, half = blocks.shape[:-1], d // group, min(d, 128)
    k = _nibbles(blocks[..., :8 * d].reshape(*lead, d // half, 16, 4, half // 32, 4))  # plane, token, c, j, code
    n = len(lead)
    k = k.permute(*range(n), n + 1, n, n + 3, n + 2, n + 4).reshape(*lead, 16, ng, group)
    # unit, g, c, word: a unit's words continue those of the one before it; a word number is (h, b, w)
    v = blocks[..., 8 * d:16 * d].reshape(*lead, d // 64, 8, 4, 16)
    v = v.permute(*range(n), n + 1, n + 2, n, n + 3).reshape(*lead, 8, 4, 2, 2, d // 64, 4)
    v = _nibbles(v)  # g, c, h, b, w, slot: token 8h + 2c + b, dimension 64w + 8 slot + g
    v = v.permute(*range(n), n + 2, n + 1, n + 3, n + 4, n + 5, n).reshape(*lead, 16, ng, group)
    meta = blocks[..., 16 * d:].contiguous().view(torch.float16).float().view(*lead, 2, 16, ng, 2)
    k = k * meta[..., 0, :, :, :1] + meta[..., 0, :, :, 1:]
    v = v * meta[..., 1, :, :, :1] + meta[..., 1, :, :, 1:]
    return k.reshape(*lead, 16, d), v.reshape(*lead, 16, d)


def _plain_attention(s):
    c = s["case"]
    h, hk, d, page = c["heads"], c["kv_heads"], c["dim"], c["page"]
    table, ctx, starts = s["table"].long(), s["ctx"].long(), s["starts"].long()
    b, width = table.shape
    blocks = s["pages"].view(-1, hk, page // 16, _block_bytes(c))[table]  # b, page, head, block, bytes
    k, v = _decode(blocks.transpose(1, 2).reshape(b, hk, -1, _block_bytes(c)), d, c["group"])
    k, v = k.reshape(b, hk, -1, d), v.reshape(b, hk, -1, d)
    n = c["q_hi"]  # queries padded to the longest
    nq = starts[1:] - starts[:-1]
    at = starts[:-1, None] + torch.arange(n, device=ctx.device)
    there = torch.arange(n, device=ctx.device) < nq[:, None]
    at = torch.where(there, at, 0)
    q = s["q"][at].float().view(b, n, hk, h // hk, d).permute(0, 2, 1, 3, 4).reshape(b, hk, n * (h // hk), d)
    x = torch.matmul(q, k.transpose(2, 3)).view(b, hk, n, h // hk, -1) * (d ** -0.5)
    key = torch.arange(width * page, device=ctx.device)
    pos = (ctx - nq)[:, None] + torch.arange(n, device=ctx.device)
    seen = key <= pos[:, :, None]
    if c["window"]:
        seen &= key > pos[:, :, None] - c["window"]
    x.masked_fill_(~seen[:, None, :, None, :], float("-inf"))
    x -= x.amax(-1, keepdim=True)
    x.exp_()
    x /= x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(b, hk, n * (h // hk), -1), v)
    o = o.view(b, hk, n, h // hk, d).permute(0, 2, 1, 3, 4).reshape(b, n, h, d)
    return o[there].bfloat16()


def _plain_rotate(x, cos, sin, rotary, interleaved):
    """x [t, heads, d] -> the same with its first `rotary` dimensions rotated, in 64 bits, rounded to 32 and then to
    x's type: codes next to a border hang on it."""
    a = x[..., :rotary].double()
    if interleaved:
        p, q = a[..., 0::2], a[..., 1::2]
    else:
        p, q = a[..., :rotary // 2], a[..., rotary // 2:]
    c, s = cos[:, None].double(), sin[:, None].double()
    u, w = p * c - q * s, q * c + p * s
    r = torch.stack((u, w), -1).flatten(-2) if interleaved else torch.cat((u, w), -1)
    return torch.cat((r.float().to(x.dtype), x[..., rotary:]), -1)


def _plain_quantize(x, group):
    """[t, heads, d] -> codes uint8 [t, heads, d], fp16 (scale, minimum) [t, heads, groups, 2]."""
    y = x.float().view(*x.shape[:2], -1, group)
    low = y.amin(-1, keepdim=True).half()
    scale = ((y.amax(-1, keepdim=True) - low.float()) / 15).half()
    n = ((y - low.float()) / scale.float()).round().clamp(0, 15)
    n = torch.where(scale == 0, 0.0, n).to(torch.uint8)
    return n.view(x.shape), torch.cat((scale, low), -1)


def _plain_places(d, ng, dev):
    """Byte offsets in a block of what token 0..15 has there: K codes and V codes [16, d / 2], scales and minima of K
    and of V [16, 4 * ng]; and the orders of the dimensions whose codes fill the bytes."""
    t = torch.arange(16, device=dev)[:, None]
    half = min(d, 128)
    i = torch.arange(d // 2, device=dev)  # plane, c, j, byte
    k_order = torch.arange(d, device=dev).view(d // half, half // 32, 4, 8).transpose(1, 2).flatten()
    k_at = (i // (half // 2)) * 8 * half + t * (half // 2) + i % (half // 2)
    v_order = torch.arange(d, device=dev).view(d // 64, 8, 8).permute(2, 0, 1).flatten()  # g, w, slot
    g, w, byte = i // (d // 16), i % (d // 16) // 4, i % 4
    word = (t // 8 * 2 + t % 2) * (d // 64) + w
    v_at = 8 * d + word // 4 * 512 + (4 * g + t % 8 // 2) * 16 + word % 4 * 4 + byte
    m = torch.arange(4 * ng, device=dev)
    return k_at, v_at, 16 * d + t * 4 * ng + m, 16 * d + 64 * ng + t * 4 * ng + m, k_order, v_order


def _plain_append(s):
    c = s["case"]
    hk, d, page, group = c["kv_heads"], c["dim"], c["page"], c["group"]
    ng, size = d // group, _block_bytes(c)
    cs = s["cos_sin"][s["positions"].long()]
    cos, sin = cs[:, :c["rotary"] // 2], cs[:, c["rotary"] // 2:]
    q = _plain_rotate(s["q"], cos, sin, c["rotary"], c["interleaved"])
    k = _plain_rotate(s["k"], cos, sin, c["rotary"], c["interleaved"])
    k_n, k_m = _plain_quantize(k, group)
    v_n, v_m = _plain_quantize(s["v"].contiguous(), group)
    k_at, v_at, km_at, vm_at, k_order, v_order = _plain_places(d, ng, q.device)
    k_n, v_n = k_n[..., k_order], v_n[..., v_order]
    slots = s["slots"]
    here = slots >= 0
    at = torch.where(here, slots, 0)
    head = torch.arange(hk, device=q.device)
    base = ((at // page)[:, None] * hk + head) * (page // 16) + (at % page // 16)[:, None]
    base, t = (base * size)[..., None], at % 16
    flat = s["pages"].view(-1)
    for where, what in ((k_at, k_n[..., 0::2] | (k_n[..., 1::2] << 4)), (v_at, v_n[..., 0::2] | (v_n[..., 1::2] << 4)),
                        (km_at, k_m.view(*k_m.shape[:2], -1).contiguous().view(torch.uint8)),
                        (vm_at, v_m.view(*v_m.shape[:2], -1).contiguous().view(torch.uint8))):
        flat[(base + where[t][:, None])[here].flatten()] = what[here].flatten()
    # what the cache now holds for these tokens; nothing for the padding
    rows = s["pages"].view(-1, hk, page // 16, size)[at // page, :, at % page // 16]
    kk, vv = _decode(rows, d, group)
    pick = t[:, None, None, None].expand(-1, hk, 1, d)
    kk, vv = (torch.where(here[:, None, None], x.gather(2, pick)[:, :, 0], 0.0).bfloat16() for x in (kk, vv))
    return q, kk, vv


def _plain_logprobs(s):
    c = s["case"]
    x, top = s["logits"], c["top"]
    m, v = x.shape
    t = s["targets"].long()[:, None]
    y = x.float() * c["scale"]
    biggest = y.amax(-1, keepdim=True)
    e = (y - biggest).exp()
    total = e.sum(-1, keepdim=True)
    lse = total.log()
    lp = y - biggest - lse
    entropy = -torch.where(e > 0, lp * e, 0.0).sum(-1) / total[:, 0]
    xt = x.gather(1, t)
    ids = torch.arange(v, device=x.device)
    rank = 1 + ((x > xt) | ((x == xt) & (ids < t))).sum(-1)
    # ties go to the lowest index: order by (value, index) as one whole number
    bits = x.float().view(torch.int32).long()
    bits = torch.where(bits < 0, -(bits & 0x7FFFFFFF), bits)  # -0.0 ties with 0.0
    _, top_ids = ((bits << 32) - ids).topk(top, -1)
    top_lp = lp.gather(1, top_ids)
    top_ids = torch.where(torch.isinf(top_lp), -1, top_ids)
    return {"logprob": lp.gather(1, t)[:, 0], "rank": rank.to(torch.int32), "entropy": entropy,
            "top_ids": top_ids.to(torch.int32), "top_logprobs": top_lp}


# ------------------------------------------------------- definition, 64 bits ----
def exact(case, seed):
    c = case
    s = prepare(case, seed)
    if c["op"] == "attention":
        return _exact_attention(c, s)
    if c["op"] == "append":
        return _exact_append(c, s)
    return _exact_logprobs(c, s)


def _exact_value(pages, c, slot, head, which):
    """Values [slots, heads, d] of K (which = 0) or V (1) at whole-cache token slots, from the place of each code."""
    d, hk, page, group = c["dim"], c["kv_heads"], c["page"], c["group"]
    ng, dev = d // group, pages.device
    slot, head = slot.view(-1, 1, 1), head.view(1, -1, 1)
    dim = torch.arange(d, device=dev).view(1, 1, -1)
    block = ((slot // page) * hk + head) * (page // 16) + slot % page // 16
    t = slot % 16
    if which == 0:
        span = min(d, 128)
        e = dim % span
        byte = dim // span * (8 * span) + t * (span // 2) + e % 32 // 8 * (span // 8) + e // 32 * 4 + e % 8 // 2
        high = e % 2
    else:
        word = (t // 8 * 2 + t % 2) * (d // 64) + dim // 64
        place = dim % 64 // 8
        byte = 8 * d + word // 4 * 512 + (4 * (dim % 8) + t % 8 // 2) * 16 + word % 4 * 4 + place // 2
        high = place % 2
    flat = pages.view(-1)
    base = block * _block_bytes(c)
    code = (flat[base + byte].long() >> (4 * high)) & 15
    halves = flat.view(torch.float16)
    meta = (base + 16 * d + which * 64 * ng + t * 4 * ng + dim // group * 4) // 2
    return halves[meta].double() * code.double() + halves[meta + 1].double()


def _exact_attention(c, s):
    ctx, nq = _lens(c)
    h, hk, d = c["heads"], c["kv_heads"], c["dim"]
    out, at = [], 0
    for b, (x, n) in enumerate(zip(ctx, nq)):
        first = max(0, x - n - c["window"] + 1) if c["window"] else 0
        key = torch.arange(first, x, device="cuda")
        slot = s["table"][b].long()[key // c["page"]] * c["page"] + key % c["page"]
        q = s["q"][at:at + n].double()
        o = torch.empty(n, h, d, dtype=torch.float64, device="cuda")
        pos = torch.arange(x - n, x, device="cuda")
        seen = key[None, :] <= pos[:, None]
        if c["window"]:
            seen &= pos[:, None] - key[None, :] < c["window"]
        for kv in range(hk):
            one = torch.tensor([kv], device="cuda")
            k = _exact_value(s["pages"], c, slot, one, 0)[:, 0]
            v = _exact_value(s["pages"], c, slot, one, 1)[:, 0]
            for j in range(kv * (h // hk), (kv + 1) * (h // hk)):
                score = (q[:, j] @ k.T) / math.sqrt(d)
                o[:, j] = torch.softmax(score.masked_fill(~seen, -math.inf), -1) @ v
        out.append(o)
        at += n
    return torch.cat(out)


def _exact_append(c, s):
    d, r = c["dim"], c["rotary"]
    table = s["cos_sin"].double()[s["positions"].long()]
    dim = torch.arange(r, device="cuda")
    if c["interleaved"]:
        other, pair, sign = dim ^ 1, dim // 2, torch.where(dim % 2 == 0, -1.0, 1.0).double()
    else:
        other, pair = (dim + r // 2) % r, dim % (r // 2)
        sign = torch.where(dim < r // 2, -1.0, 1.0).double()
    cos, sin = table[:, None, pair], table[:, None, r // 2 + pair] * sign

    def turned(x):
        y = x.double()
        y[..., :r] = y[..., :r] * cos + y[..., other] * sin
        return y

    def held(x):  # the cache's definition: every step rounded as it names
        y = x.float().reshape(*x.shape[:2], d // c["group"], c["group"])
        low = y.min(-1, keepdim=True).values.half().float()
        step = ((y.max(-1, keepdim=True).values - low) / 15.0).half().float()
        n = torch.where(step > 0, ((y - low) / step).round(), torch.zeros_like(y)).clamp(0, 15)
        z = n.double() * step.double() + low.double()
        return torch.where((s["slots"] >= 0)[:, None, None], z.reshape(x.shape), 0.0)

    return turned(s["q"]), held(turned(s["k"]).float().bfloat16()), held(s["v"])


def _exact_logprobs(c, s):
    x, top = s["logits"], c["top"]
    m, v = x.shape
    lp, ent, top_lp = (torch.empty(m, dtype=torch.float64, device="cuda"),
                       torch.empty(m, dtype=torch.float64, device="cuda"),
                       torch.empty(m, top, dtype=torch.float64, device="cuda"))
    for i in range(0, m, 64):
        y = torch.log_softmax(x[i:i + 64].double() * c["scale"], -1)
        lp[i:i + 64] = y.gather(1, s["targets"][i:i + 64].long()[:, None])[:, 0]
        ent[i:i + 64] = -torch.special.xlogy(y.exp(), y.exp()).sum(-1)
        top_lp[i:i + 64] = y.sort(-1, descending=True).values[:, :top]
    return {"logprob": lp, "rank": None, "entropy": ent, "top_ids": None, "top_logprobs": top_lp}
