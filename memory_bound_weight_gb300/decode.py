"""A whole decode step: the weight-streaming products with the 4-bit cache and
its attention between them and the tokens' log probabilities behind them.

    python -m memory_bound_weight_gb300.decode --model tinyllama --layers 22 --requests 4 --prompt 200 --tokens 64

Random weights of a workload's shapes (no checkpoint is needed), greedy
decoding of a few requests whose prompts differ in length. Per layer:

    qkv = W_qkv . norm(x)            gemv_fused (RMSNorm prologue)
    q, cache <- qkv                  kv4_append (rotation, 4-bit keys and values)
    a = attention(q, cache)          kv4_attention
    x = x + W_o . a                  gemv_fused (residual epilogue)
    x = x + W_down . (silu(W_gate . norm(x)) * (W_up . norm(x)))   two gemv_fused

and behind the last one logits = W_head . norm(x) and token_logprobs. A step for
one token of every request is captured into a CUDA graph and replayed: the
lengths, positions and slots it works on are device tensors that it moves on
itself. (The length of a shared beginning, below, is not: a captured step is
refused behind prompts that share less.)

With --weights fp8 each product is one of 8-bit floating point operands with a
scale for each block of 128: quantize_fp8_g128 (with the norm where there is one)
and gemm_fp8_b128, gate and up in one call. With --shared N the requests' prompts
begin with the same N tokens, whose keys and values are computed and held once;
attention is then kv4_attention_shared (whose workspace is sized for a step's
tokens: the rest of the prompts, in one pass, reads the shared pages for each request).
"""
from __future__ import annotations

import argparse
from dataclasses import dataclass

import torch

import memory_bound_weight_gb300 as mbw


@dataclass(frozen=True)
class Shape:
    hidden: int
    heads: int
    kv_heads: int
    dim: int
    mlp: int
    vocab: int
    layers: int
    rope_base: float


# The decode workloads of workloads.py, with their head layouts.
SHAPES = {
    "tinyllama": Shape(2048, 32, 4, 64, 5632, 32000, 22, 1e4),
    "qwen25-7b": Shape(3584, 28, 4, 128, 18944, 152064, 28, 1e6),
    "qwen3-4b": Shape(2560, 32, 8, 128, 9728, 151936, 36, 1e6),
}


class Decoder:
    """Weights (bf16, or fp8: 8-bit floating point with a scale for each block of 128), caches and buffers for up to
    `requests` requests of up to `max_tokens` tokens each."""

    shared = 0  # tokens that all requests begin with, in the same pages
    fp8 = False

    def __init__(self, shape, layers=None, requests=1, max_tokens=1024, page_size=16, group=64, seed=0, weights="bf16"):
        if weights not in ("bf16", "fp8"):
            raise ValueError(f"weights must be bf16 or fp8, got {weights}")
        self.shape, self.requests, self.fp8 = shape, requests, weights == "fp8"
        n = shape.layers if layers is None else layers
        s, dev = shape, "cuda"
        gen = torch.Generator(device=dev)
        gen.manual_seed(seed)

        def plain(rows, cols):
            return (torch.randn(rows, cols, generator=gen, device=dev) * cols ** -0.5).bfloat16()

        def weight(rows, cols):
            w = plain(rows, cols)
            return mbw.quantize_fp8_b128(w) if self.fp8 else w

        def ones(width):
            return (1 + 0.1 * torch.randn(width, generator=gen, device=dev)).bfloat16()

        width = (s.heads + 2 * s.kv_heads) * s.dim
        self.layers = [dict(norm1=ones(s.hidden), qkv=weight(width, s.hidden), o=weight(s.hidden, s.heads * s.dim),
                            norm2=ones(s.hidden), gate=weight(s.mlp, s.hidden), up=weight(s.mlp, s.hidden),
                            down=weight(s.hidden, s.mlp)) for _ in range(n)]
        self.embedding, self.norm, self.head = plain(s.vocab, s.hidden), ones(s.hidden), weight(s.vocab, s.hidden)
        self.embedding *= s.hidden ** 0.5
        # each request has its own pages, the same ones in every layer's cache, in no particular order
        per = -(-max_tokens // page_size)
        self.page_size, self.max_tokens = page_size, max_tokens
        self.table = torch.randperm(requests * per, generator=gen, device=dev).to(torch.int32).view(requests, per)
        size = mbw.kv4_page_bytes(page_size, s.kv_heads, s.dim, group)
        self.caches = [mbw.Kv4Cache(torch.empty(requests * per, size, dtype=torch.uint8, device=dev), s.kv_heads, s.dim,
                                    page_size, group) for _ in range(n)]
        self.cos_sin = mbw.rope_table(max_tokens, s.dim, s.rope_base)
        self.ctx = torch.zeros(requests, dtype=torch.int32, device=dev)  # tokens in the cache
        self.ids = torch.zeros(requests, dtype=torch.int64, device=dev)  # the next ones
        self.longest = 0  # the largest of ctx, known on the host: a step past max_tokens would index past the tables
        self.own_table = self.table.clone()
        self.attn_ws = mbw.kv4_attention_shared_workspace(s.dim, requests, s.heads)
        self.prob_ws = mbw.token_logprobs_workspace()

    def tune(self, rows=None):
        """Measures the products' plans for `rows` tokens (those of a step by default). Those of 8 bits have none."""
        if self.fp8:
            return
        s, m, op = self.shape, rows or self.requests, mbw.OP_GEMV_BF16
        for fuse, n, k in ((mbw.FUSE_NORM, (s.heads + 2 * s.kv_heads) * s.dim, s.hidden),
                           (mbw.FUSE_RESIDUAL, s.hidden, s.heads * s.dim),
                           (mbw.FUSE_NORM | mbw.FUSE_GLU, s.mlp, s.hidden), (mbw.FUSE_RESIDUAL, s.hidden, s.mlp),
                           (mbw.FUSE_NORM, s.vocab, s.hidden)):
            mbw.autotune(op | fuse, m, n, k)

    def product(self, w, x, norm=None, up=None, residual=None):
        """x . w^T (+ residual) of the normed x; with `up`, silu(x . w^T) * (x . up^T)."""
        if self.fp8:
            q, scales = mbw.quantize_fp8_g128(x, norm_weight=norm)
            u, us = up or (None, None)
            return mbw.gemm_fp8_b128(q, scales, *w, residual=residual, up_weights=u, up_scales=us)
        return mbw.gemv_fused(mbw.OP_GEMV_BF16, w, None, x, norm_weight=norm, up_weights=up, residual=residual)

    def attend(self, cache, q, q_starts):
        if self.shared:
            return mbw.kv4_attention_shared(cache, q, self.table, self.ctx, self.shared, q_starts, workspace=self.attn_ws)
        return mbw.kv4_attention(cache, q, self.table, self.ctx, q_starts, workspace=self.attn_ws)

    def forward(self, ids, request, positions, q_starts, last):
        """Tokens `ids` at `positions` of the requests `request` (each a tensor (T,), a request's tokens together) through
        the layers; self.ctx counts them already. Returns the logits of the tokens `last`, none for None."""
        s = self.shape
        T = ids.shape[0]
        page = self.table[request, positions // self.page_size].long()
        slots, pos32 = page * self.page_size + positions % self.page_size, positions.to(torch.int32)
        x = self.embedding[ids]
        for w, cache in zip(self.layers, self.caches):
            qkv = self.product(w["qkv"], x, norm=w["norm1"]).view(T, -1, s.dim)
            q, k, v = qkv.split((s.heads, s.kv_heads, s.kv_heads), 1)
            mbw.kv4_append(cache, k, v, slots, q=q, positions=pos32, cos_sin=self.cos_sin, q_out=q)
            a = self.attend(cache, q, q_starts)
            x = self.product(w["o"], a.view(T, -1), residual=x)
            g = self.product(w["gate"], x, norm=w["norm2"], up=w["up"])
            x = self.product(w["down"], g, residual=x)
        return None if last is None else self.product(self.head, x[last], norm=self.norm)

    def prompt(self, prompts, share=False):
        """Fills the caches with the prompts (one list of ids per request) and returns their last logits' TokenLogprobs.
        share: what they have in common at their beginning, in whole pages, is computed and held once, and the steps that
        follow attend to it once for all requests."""
        dev = self.ids.device
        n = [len(p) for p in prompts]
        if len(n) != self.requests:
            raise ValueError(f"{self.requests} prompts are needed, got {len(n)}")
        if min(n) < 1:
            raise ValueError("a prompt is empty")
        if max(n) > self.max_tokens:
            raise ValueError(f"a prompt of {max(n)} tokens is longer than max_tokens, {self.max_tokens}")
        if any(not 0 <= t < self.shape.vocab for p in prompts for t in p):
            raise ValueError(f"a prompt has an id outside 0 to {self.shape.vocab - 1}")
        if self.shared:  # every request in its own pages again
            self.table.copy_(self.own_table)
            self.shared = 0
        common = self.common(prompts) if share else 0
        if common:  # as tokens of the first request, whose pages the others' tables then name
            self.table[:, :common // self.page_size] = self.table[:1, :common // self.page_size].clone()
            self.ctx.zero_()
            self.ctx[:1] = common
            at = torch.arange(common, device=dev)
            try:
                self.forward(torch.tensor(prompts[0][:common], device=dev), torch.zeros_like(at), at,
                             torch.tensor([0] + [common] * len(n), dtype=torch.int32, device=dev), None)
            except BaseException:  # nobody shares what is not there: the next prompts find each request in its own pages
                self.table.copy_(self.own_table)
                raise
            self.shared = common
        starts = [0]
        for x in n:
            starts.append(starts[-1] + x - common)
        ids = torch.tensor([t for p in prompts for t in p[common:]], device=dev)
        request = torch.repeat_interleave(torch.arange(len(n), device=dev), torch.tensor(n, device=dev) - common)
        positions = torch.cat([torch.arange(common, x, device=dev) for x in n])
        self.ctx.copy_(torch.tensor(n, dtype=torch.int32))
        self.longest = max(n)
        logits = self.forward(ids, request, positions, torch.tensor(starts, dtype=torch.int32, device=dev),
                              torch.tensor(starts[1:], device=dev) - 1)
        return self.choose(logits)

    def common(self, prompts):
        """Tokens that all prompts begin with, in whole pages; each has one more at least."""
        most = min(len(p) for p in prompts) - 1
        same = next((i for i in range(most) if any(p[i] != prompts[0][i] for p in prompts)), most)
        return same // self.page_size * self.page_size

    def advance(self):
        """Counts a token more on the host, or raises where the longest request has no place for it."""
        if self.longest >= self.max_tokens:
            raise ValueError(f"a request has max_tokens, {self.max_tokens}, already")
        self.longest += 1

    def step(self, top_k=1):
        """One token of every request: self.ids go in at their places, and the most likely next ones take theirs."""
        self.advance()
        positions = self.ctx.long()
        self.ctx += 1
        return self.choose(self.forward(self.ids, torch.arange(self.requests, device=positions.device), positions, None,
                                        slice(None)), top_k)

    def choose(self, logits, top_k=1):
        r = mbw.token_logprobs(logits, top_k=top_k, workspace=self.prob_ws)
        self.ids.copy_(r.top_ids[:, 0])
        return r

    def counted(self, replay):
        """A captured step as a call. It holds the number of tokens that the requests shared when it was captured; with fewer, or
        none, it would have them attend to another's pages. (With more it attends to the others as to each request's own.)"""
        shared = self.shared

        def counted_replay():
            if shared > self.shared:
                raise ValueError(f"captured for {shared} tokens that all requests share, which now share {self.shared}: capture anew")
            self.advance()
            replay()

        return counted_replay

    def graph(self, top_k=1):
        """step() as a CUDA graph: (replay, its TokenLogprobs, overwritten by each replay). One place has to be left. Replays
        follow further prompts, but for those that share fewer tokens than when it was captured, behind which they raise."""
        keep, longest = (self.ctx.clone(), self.ids.clone()), self.longest
        self.advance()  # refused before anything runs
        self.longest = longest
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            self.step(top_k)  # plans and allocations happen here
            side.synchronize()
            self.longest = longest
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=side):
                out = self.step(top_k)
        torch.cuda.current_stream().wait_stream(side)
        self.ctx.copy_(keep[0])
        self.ids.copy_(keep[1])
        self.longest = longest
        return self.counted(g.replay), out


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--model", choices=sorted(SHAPES), default="tinyllama")
    ap.add_argument("--layers", type=int, default=None, help="fewer than the model has")
    ap.add_argument("--requests", type=int, default=1)
    ap.add_argument("--prompt", type=int, default=128, help="tokens of the longest prompt")
    ap.add_argument("--tokens", type=int, default=64)
    ap.add_argument("--weights", choices=("bf16", "fp8"), default="bf16")
    ap.add_argument("--shared", type=int, default=0, help="tokens in front of every prompt, the same ones")
    a = ap.parse_args()
    shape = SHAPES[a.model]
    d = Decoder(shape, a.layers, a.requests, max_tokens=a.shared + a.prompt + a.tokens + 2, weights=a.weights)
    gen = torch.Generator().manual_seed(1)
    prompts = [torch.randint(shape.vocab, (max(1, a.prompt - 7 * i),), generator=gen).tolist() for i in range(a.requests)]
    if a.shared:
        front = torch.randint(shape.vocab, (a.shared,), generator=gen).tolist()
        prompts = [front + p for p in prompts]
    d.tune()
    d.prompt(prompts, share=a.shared > 0)
    replay, out = d.graph(top_k=5)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    torch.cuda.synchronize()
    start.record()
    for _ in range(a.tokens):
        replay()
    end.record()
    end.synchronize()
    ms = start.elapsed_time(end) / a.tokens
    print(f"{a.model}, {len(d.layers)} layers, {a.requests} request(s), context {int(d.ctx.max())}: {ms:.3f} ms per step, "
          f"{a.requests * 1e3 / ms:.0f} tokens/s")
    for i in range(min(a.requests, 4)):
        print(f"request {i}: entropy {out.entropy[i].item():.3f}, top " +
              ", ".join(f"{t} ({p:.3f})" for t, p in zip(out.top_ids[i].tolist(), out.top_logprobs[i].tolist())))
    mbw.check_device_error()


if __name__ == "__main__":
    main()
