"""Measured cases of the operators for serving a batch of requests behind one
long prompt: products in 8-bit floating point with a scale for each block of 128
(plain, and the gated form of a feed-forward block), the quantization of their
operands, and attention over the 4-bit paged cache for a batch whose requests
share a prefix.

Each case is one call as a serving engine makes it. ``run`` computes it in its
plain form (elementary torch operations, 32 bits) or, with ``own`` set, through
the package's entry points. ``exact`` is the operators' definition in 64 bits.

An 8-bit value is an e4m3 code times an fp32 scale: one scale per row and 128
columns of the activations, one per 128 x 128 of the weights. The scale is the
largest magnitude divided by 448, the code the value divided by the scale, both
divisions IEEE fp32, rounded to nearest even.
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
LAYOUTS = (QWEN25, TINYLLAMA, QWEN3, QWEN3, WIDE)

# Their matrices (outputs, inputs): QKV, attention output, gate or up, down.
MATRICES = ((4608, 3584), (3584, 3584), (18944, 3584), (3584, 18944),
            (2560, 2048), (2048, 2048), (5632, 2048), (2048, 5632),
            (6144, 2560), (2560, 4096), (9728, 2560), (2560, 9728))


def _product(name, m, n, k, gated=False, residual=False):
    return {"name": name, "op": "gated" if gated else "product", "m": m, "n": n, "k": k, "residual": residual}


def _quantize(name, m, k, what="tokens", norm=False):
    return {"name": name, "op": "quantize", "what": what, "m": m, "k": k, "norm": norm}


def _shared(name, layout, batch, prefix, lo, hi, q_lo=1, q_hi=1, page=16, group=64, window=0):
    return {"name": name, "op": "shared", **layout, "batch": batch, "prefix": prefix, "own_lo": lo, "own_hi": hi,
            "q_lo": q_lo, "q_hi": q_hi, "page": page, "group": group, "window": window}


def listed():
    return [
        # one token of a small model, attention output: latency alone
        _product("product 1x2048x2048", 1, 2048, 2048, residual=True),
        # a decode step of a small batch, the down projection into the residual stream
        _product("product 16x3584x18944", 16, 3584, 18944, residual=True),
        # the last chunk of a prompt, QKV
        _product("product 777x4608x3584", 777, 4608, 3584),
        # a long prompt, the down projection
        _product("product 4096x3584x18944", 4096, 3584, 18944, residual=True),
        # one token, both projections of the feed-forward block
        _product("gated 1x18944x3584", 1, 18944, 3584, gated=True),
        # a decode step of a full batch
        _product("gated 61x5632x2048", 61, 5632, 2048, gated=True),
        # a prompt
        _product("gated 2048x9728x2560", 2048, 9728, 2560, gated=True),
        # one token's hidden state in front of a projection
        _quantize("quantize tokens 1x3584 norm", 1, 3584, norm=True),
        # a prompt's hidden states
        _quantize("quantize tokens 4000x3584 norm", 4000, 3584, norm=True),
        # the load-time step of one matrix
        _quantize("quantize weights 18944x3584", 18944, 3584, "weights"),
        # a full batch behind a long system prompt, one token each
        _shared("shared 64x1 prefix 8192", QWEN3, 64, 8192, 20, 900, page=32),
        # verification of drafted tokens behind a document
        _shared("shared 12x(2-5) prefix 30000", QWEN25, 12, 30000, 40, 700, 2, 5, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(("product", "product", "gated", "quantize", "shared", "shared"))
    if op in ("product", "gated"):
        n, k = rng.choice(MATRICES)
        if rng.random() < 0.4:  # any width, any number of blocks
            n, k = _log(rng, 64, 19000), 128 * _log(rng, 1, 148)
        most = 4096 * 3584 * 18944 // (n * k * (2 if op == "gated" else 1))
        m = _log(rng, 1, max(1, min(4096, most)))
        c = _product("", m, n, k, op == "gated", rng.random() < 0.5)
    elif op == "quantize":
        what = rng.choice(("tokens", "tokens", "weights"))
        k = 128 * _log(rng, 1, 148)
        m = _log(rng, 1, min(20_000, 67_000_000 // k))
        c = _quantize("", m, k, what, what == "tokens" and rng.random() < 0.5)
    else:
        layout = rng.choice(LAYOUTS)
        batch = _log(rng, 2, 130)
        prefix = _log(rng, 64, 30_000)
        most = rng.choice((1, 1, 1, 8, 100))
        q_hi = rng.randint(1, max(1, min(most, 500 // batch)))
        q_lo = rng.randint(1, q_hi)
        # the plain form holds the scores of all rows and keys at once
        prefix = max(64, min(prefix, 600_000_000 // (batch * q_hi * layout["heads"])))
        hi = _log(rng, max(8, q_hi), max(q_hi, min(2000, 200_000_000 // (batch * q_hi * layout["heads"]))))
        hi = max(hi, q_hi)
        lo = rng.randint(max(1, hi // 40), hi)
        c = _shared("", layout, batch, prefix, lo, hi, q_lo, q_hi, rng.choice((16, 32, 64)), rng.choice((32, 64)),
                    rng.choice((0, 0, 0, rng.randint(64, 8192))))
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
    """Tokens of each request behind the prefix, and how many of them are queries."""
    mine = _spread(c["own_lo"], c["own_hi"], c["batch"], 0.31)
    nq = _spread(c["q_lo"], c["q_hi"], c["batch"], 0.77)
    return mine, [min(n, x) for n, x in zip(nq, mine)]


def _block_bytes(c):
    return 16 * c["dim"] + 128 * (c["dim"] // c["group"])


def work(case):
    c = case
    if c["op"] in ("product", "gated"):
        m, n, k = c["m"], c["n"], c["k"]
        kb, nb, w = k // 128, -(-n // 128), 2 if c["op"] == "gated" else 1
        return {"bytes": m * (k + 4 * kb) + w * (n * k + 4 * nb * kb) + 2 * m * n * (2 if c["residual"] else 1),
                "flops": 2 * w * m * n * k}
    if c["op"] == "quantize":
        m, k = c["m"], c["k"]
        scales = 4 * (k // 128) * (m if c["what"] == "tokens" else -(-m // 128))
        # read, codes and scales written; codes and scales read back, values written
        return {"bytes": m * k * (2 + 1 + 1 + 4) + 2 * scales + (2 * k if c["norm"] else 0), "flops": 6 * m * k}
    mine, nq = _lens(c)
    p, w, per_token = c["prefix"], c["window"], c["dim"] + 8 * (c["dim"] // c["group"])
    keys, pairs = 0, 0
    once = max((min(p, w + n - x - 1) if w else p) for x, n in zip(mine, nq))  # prefix tokens that some query sees
    for x, n in zip(mine, nq):
        keys += min(x, w + n - 1) if w else x
        for i in range(p + x - n, p + x):
            pairs += min(i + 1, w) if w else i + 1
    rows = sum(nq) * c["heads"]
    return {"bytes": (max(0, once) + keys) * c["kv_heads"] * per_token + 4 * rows * c["dim"],
            "flops": 4 * pairs * c["heads"] * c["dim"]}


# ----------------------------------------------------------------- inputs ----
def _e4m3(x, scale):
    return torch.where(scale > 0, x / scale, torch.zeros_like(x)).to(torch.float8_e4m3fn)


def _scale(high):  # by a tensor: torch multiplies by the reciprocal of a number
    return high / torch.full_like(high, 448.0)


def _by_rows(x):
    """Codes and scales of bf16 or fp32 rows, a scale per 128 columns."""
    m, k = x.shape
    y = x.float().view(m, k // 128, 128)
    scale = _scale(y.abs().amax(-1))
    return _e4m3(y, scale[..., None]).view(m, k), scale


def _by_blocks(w):
    """Codes and scales of a matrix, a scale per 128 x 128; the last rows may be fewer."""
    n, k = w.shape
    codes = torch.empty(n, k, dtype=torch.float8_e4m3fn, device=w.device)
    scales = torch.empty(-(-n // 128), k // 128, dtype=torch.float32, device=w.device)
    for i in range(0, n, 1024):
        y = w[i:i + 1024].float()
        rows = y.shape[0]
        y = torch.nn.functional.pad(y, (0, 0, 0, -rows % 128)).view(-1, 128, k // 128, 128)
        s = _scale(y.abs().amax((1, 3)))
        scales[i // 128:i // 128 + s.shape[0]] = s
        codes[i:i + 1024] = _e4m3(y, s[:, None, :, None]).view(-1, k)[:rows]
    return codes, scales


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dev = "cuda"

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    def uniform(lo, hi, *shape):
        return torch.rand(*shape, generator=g, device=dev, dtype=torch.float32) * (hi - lo) + lo

    def hidden(m, k):  # channels of unequal size, a few of them far larger, as hidden states have
        size = torch.exp(normal(k) * 0.6)
        size[torch.randint(k, (max(1, k // 500),), generator=g, device=dev)] *= 25
        return (normal(m, k) * size).bfloat16()

    def weights(n, k):
        w = torch.empty(n, k, dtype=torch.bfloat16, device=dev)
        for i in range(0, n, 4096):
            rows = min(n, i + 4096) - i
            w[i:i + rows] = normal(rows, k) * k ** -0.5 * uniform(0.5, 1.5, rows, 1)
        return w

    s = {"case": dict(c)}
    if c["op"] in ("product", "gated"):
        s["x"], s["x_scales"] = _by_rows(hidden(c["m"], c["k"]))
        s["w"], s["w_scales"] = _by_blocks(weights(c["n"], c["k"]))
        if c["op"] == "gated":
            s["up"], s["up_scales"] = _by_blocks(weights(c["n"], c["k"]))
        s["residual"] = hidden(c["m"], c["n"]) if c["residual"] else None
        s["workspace"] = torch.zeros(64 << 20, dtype=torch.uint8, device=dev)
    elif c["op"] == "quantize":
        if c["what"] == "weights":
            s["x"] = weights(c["m"], c["k"])
        else:
            s["x"] = hidden(c["m"], c["k"])
        s["norm"] = (1 + 0.1 * normal(c["k"])).bfloat16() if c["norm"] else None
    else:
        mine, nq = _lens(c)
        hk, d, page, p = c["kv_heads"], c["dim"], c["page"], c["prefix"]
        ng, blocks = d // c["group"], page // 16
        common = p // page  # whole pages; what is left of the prefix lies in each request's own pages
        used = [-(-(p + x) // page) - common for x in mine]
        pages = common + sum(used) + 3
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
        order = torch.randperm(pages, generator=g, device=dev).to(torch.int32).cpu()
        table, at = torch.zeros(c["batch"], common + max(used), dtype=torch.int32), common
        table[:, :common] = order[:common]
        for b, u in enumerate(used):
            table[b, common:common + u] = order[at:at + u]
            at += u
        s["table"] = table.cuda()
        s["ctx"] = torch.tensor([p + x for x in mine], dtype=torch.int32, device=dev)
        starts = [0]
        for x in nq:
            starts.append(starts[-1] + x)
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
        # the query part of the projections' output: rows of a wider matrix
        wide = (normal(starts[-1], (c["heads"] + 2 * hk) * d) * 2).bfloat16()
        s["q"] = wide[:, :c["heads"] * d].view(starts[-1], c["heads"], d)
        s["workspace"] = torch.zeros(64 << 20, dtype=torch.uint8, device=dev)
    return s


# ---------------------------------------------------------------- running ----
def run(state):
    op = state["case"]["op"]
    if own:
        return _own(state, op)
    return {"product": _plain_product, "gated": _plain_product, "quantize": _plain_quantize,
            "shared": _plain_shared}[op](state)


def _own(s, op):
    import memory_bound_weight_gb300 as mbw

    c = s["case"]
    if op in ("product", "gated"):
        return mbw.gemm_fp8_b128(s["x"], s["x_scales"], s["w"], s["w_scales"], residual=s["residual"],
                                 up_weights=s.get("up"), up_scales=s.get("up_scales"), workspace=s["workspace"])
    if op == "quantize":  # the codes, read back as the values they stand for
        if c["what"] == "weights":
            codes, scales = mbw.quantize_fp8_b128(s["x"])
            return mbw.dequant_fp8_b128(codes, scales), scales
        codes, scales = mbw.quantize_fp8_g128(s["x"], norm_weight=s["norm"], norm_eps=1e-6)
        return mbw.dequant_fp8_g128(codes, scales), scales
    cache = mbw.Kv4Cache(s["pages"], c["kv_heads"], c["dim"], c["page"], c["group"])
    return mbw.kv4_attention_shared(cache, s["q"], s["table"], s["ctx"], c["prefix"],
                                    s["starts"] if c["q_hi"] > 1 else None, window=c["window"],
                                    workspace=s["workspace"])


def _matrix(codes, scales):
    """fp32 values of a matrix held with a scale per 128 x 128."""
    n, k = codes.shape
    wide = scales.repeat_interleave(128, 0)[:n]
    return (codes.float().view(n, k // 128, 128) * wide[:, :, None]).view(n, k)


def _plain_product(s):
    m, k = s["x"].shape
    x = (s["x"].float().view(m, k // 128, 128) * s["x_scales"][:, :, None]).view(m, k)
    y = torch.matmul(x, _matrix(s["w"], s["w_scales"]).t())
    if s["case"]["op"] == "gated":
        y = y / (1 + torch.exp(-y)) * torch.matmul(x, _matrix(s["up"], s["up_scales"]).t())
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return y.bfloat16()


def _plain_quantize(s):
    x, c = s["x"], s["case"]
    if c["what"] == "weights":
        codes, scales = _by_blocks(x)
        return _matrix(codes, scales), scales
    y = x.float()
    if c["norm"]:  # the mean in 64 bits: its factor decides roundings of every value of the row
        r = (1 / torch.sqrt(x.double().square().mean(-1, keepdim=True) + 1e-6)).float()
        y = (y * r * s["norm"].float()).bfloat16().float()
    codes, scales = _by_rows(y)
    m, k = codes.shape
    return (codes.float().view(m, k // 128, 128) * scales[:, :, None]).view(m, k), scales


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


def _plain_shared(s):
    c = s["case"]
    h, hk, d, page = c["heads"], c["kv_heads"], c["dim"], c["page"]
    gq, common = h // hk, c["prefix"] // page
    table, ctx, starts = s["table"].long(), s["ctx"].long(), s["starts"].long()
    b = table.shape[0]
    paged = s["pages"].view(-1, hk, page // 16, _block_bytes(c))
    # the common pages once, the rest per request
    kp, vp = _decode(paged[table[0, :common]].transpose(0, 1).reshape(hk, -1, _block_bytes(c)), d, c["group"])
    kp, vp = kp.reshape(hk, -1, d), vp.reshape(hk, -1, d)
    ko, vo = _decode(paged[table[:, common:]].transpose(1, 2).reshape(b, hk, -1, _block_bytes(c)), d, c["group"])
    ko, vo = ko.reshape(b, hk, -1, d), vo.reshape(b, hk, -1, d)
    n = c["q_hi"]  # queries padded to the longest
    nq = starts[1:] - starts[:-1]
    at = starts[:-1, None] + torch.arange(n, device=ctx.device)
    there = torch.arange(n, device=ctx.device) < nq[:, None]
    at = torch.where(there, at, 0)
    q = s["q"][at].float().view(b, n, hk, gq, d).permute(0, 2, 1, 3, 4) * (d ** -0.5)  # b, head, query, of group, d
    xp = torch.matmul(q.permute(1, 0, 2, 3, 4).reshape(hk, b * n * gq, d), kp.transpose(1, 2))
    xp = xp.view(hk, b, n, gq, common * page).transpose(0, 1)
    xo = torch.matmul(q.reshape(b, hk, n * gq, d), ko.transpose(2, 3)).view(b, hk, n, gq, -1)
    pos = (ctx - nq)[:, None] + torch.arange(n, device=ctx.device)

    def mask(x, key):
        seen = key <= pos[:, :, None]
        if c["window"]:
            seen &= key > pos[:, :, None] - c["window"]
        return x.masked_fill(~seen[:, None, :, None, :], float("-inf"))

    xp = mask(xp, torch.arange(common * page, device=ctx.device))
    xo = mask(xo, common * page + torch.arange(xo.shape[-1], device=ctx.device))
    top = xo.amax(-1, keepdim=True)
    if common:
        top = torch.maximum(top, xp.amax(-1, keepdim=True))
    xp, xo = torch.exp(xp - top), torch.exp(xo - top)
    total = xp.sum(-1, keepdim=True) + xo.sum(-1, keepdim=True)
    o = torch.matmul(xo.view(b, hk, n * gq, -1), vo).view(b, hk, n, gq, d)
    op = torch.matmul(xp.transpose(0, 1).reshape(hk, b * n * gq, -1), vp).view(hk, b, n, gq, d)
    o = (o + op.transpose(0, 1)) / total
    return o.permute(0, 2, 1, 3, 4).reshape(b, n, h, d)[there].bfloat16()


# ------------------------------------------------------------------ exact ----
def exact(case, seed):
    s = prepare(case, seed)
    return {"product": _exact_product, "gated": _exact_product, "quantize": _exact_quantize,
            "shared": _exact_shared}[case["op"]](case, s)


def _exact_product(c, s):
    k, n = c["k"], c["n"]

    def product(codes, scales):  # a block of 128 inputs at a time, the scales applied to its sums
        y = torch.zeros(c["m"], n, dtype=torch.float64, device="cuda")
        row = torch.arange(n, device="cuda") // 128
        for i in range(k // 128):
            cut = slice(128 * i, 128 * i + 128)
            part = s["x"][:, cut].double() @ codes[:, cut].double().T
            y += part.mul_(s["x_scales"][:, i, None].double()).mul_(scales[row, i].double())
        return y

    y = product(s["w"], s["w_scales"])
    if c["op"] == "gated":
        y = y * torch.sigmoid(y) * product(s["up"], s["up_scales"])
    return y if s["residual"] is None else y + s["residual"].double()


def _exact_quantize(c, s):
    """The definition, every step rounded as it names: the norm's factor to fp32, its products to fp32 and bf16, the scale
    and the quotient to fp32, the code to e4m3; the value is the code times the scale."""
    x = s["x"]
    if c["norm"]:
        f = torch.rsqrt((x.double() * x.double()).sum(1) / c["k"] + 1e-6).float()
        x = ((x.float() * f[:, None]) * s["norm"].float()).bfloat16()
    high = torch.stack([p.float().abs().amax(1) for p in x.split(128, 1)], 1)
    if c["what"] == "weights":
        high = torch.stack([p.amax(0) for p in high.split(128, 0)])
    scale = (high.double() / 448.0).float()  # 53 bits and then 24: the quotient of fp32 numbers, correctly rounded
    full = scale if c["what"] == "tokens" else scale.repeat_interleave(128, 0)[:c["m"]]
    out = torch.empty(c["m"], c["k"], dtype=torch.float64, device="cuda")
    for i in range(c["k"] // 128):
        cut, f = slice(128 * i, 128 * i + 128), full[:, i, None]
        code = torch.where(f > 0, x[:, cut].float() / f, 0.0).double()
        # to e4m3: three bits behind the leading one, down to 2^-9
        step = torch.exp2(torch.clamp(torch.floor(torch.log2(code.abs().clamp_min(1e-30))), min=-6) - 3)
        out[:, cut] = (code / step).round() * step * f.double()
    return out, scale.double()


def _exact_shared(c, s):
    """Request by request, over all of its keys."""
    h, hk, d, page, w = c["heads"], c["kv_heads"], c["dim"], c["page"], c["window"]
    starts, ctx = s["starts"].tolist(), s["ctx"].tolist()
    out = torch.empty(starts[-1], h, d, dtype=torch.float64, device="cuda")
    for b, length in enumerate(ctx):
        ids = s["table"][b, :-(-length // page)].long()
        raw = s["pages"][ids].view(len(ids), hk, page // 16, -1).permute(1, 0, 2, 3).reshape(hk, -1, _block_bytes(c))
        k, v = (x.reshape(hk, -1, d)[:, :length].double() for x in _exact_values(raw, d, c["group"]))
        a, e = starts[b], starts[b + 1]
        n = e - a
        q = s["q"][a:e].double().view(n, hk, h // hk, d)
        x = torch.einsum("nkgd,ktd->nkgt", q, k) / math.sqrt(d)
        t = torch.arange(length, device="cuda")
        p = torch.arange(length - n, length, device="cuda")[:, None]
        hide = (t > p) | (t <= p - w) if w else t > p
        x = torch.softmax(x.masked_fill(hide[:, None, None], -math.inf), -1)
        out[a:e] = torch.einsum("nkgt,ktd->nkgd", x, v).reshape(n, h, d)
    return out


def _exact_values(raw, d, group):
    """K and V of blocks, by the place of each value: the word that holds it and the code in the word."""
    t, e = torch.arange(16, device="cuda")[:, None], torch.arange(d, device="cuda")[None]
    span = min(d, 128)
    ke = e % span
    k_byte = e // span * 8 * span + t * (span // 2) + ke % 32 // 8 * (span // 8) + ke // 32 * 4 + ke % 8 // 2
    word = ((t // 8) * 2 + t % 2) * (d // 64) + e // 64
    slot = e % 64 // 8
    v_byte = 8 * d + word // 4 * 512 + (4 * (e % 8) + t % 8 // 2) * 16 + word % 4 * 4 + slot // 2
    meta = raw[..., 16 * d:].contiguous().view(torch.float16).double().view(*raw.shape[:-1], 2, 16, d // group, 2)
    out = []
    for i, (at, odd) in enumerate(((k_byte, ke % 2), (v_byte, slot % 2))):
        code = (raw[..., at.expand(16, d).long()] >> (4 * odd).to(torch.uint8)) & 15
        pair = meta[..., i, :, :, :].repeat_interleave(group, -2)
        out.append(code.double() * pair[..., 0] + pair[..., 1])
    return out
