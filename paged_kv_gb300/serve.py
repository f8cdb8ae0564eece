"""A small decoder served end to end through the library's calls.

``python -m paged_kv_gb300.serve [requests] [new_tokens]`` serves random prompts
(default 8 requests, 16 new tokens each) with random weights and prints the
tokens of the first requests.  ``Engine`` is the example to read: one step is

    prepare_step     pages for the new positions; packed positions, ids, locations
    append_kv        each layer's new keys and values, rotated, into its cache
    paged_attention  each layer's new queries over its cache
    adjust_logits    penalties, biases and a grammar mask on the last rows' logits
    sample_batch     one token a row, written back into the token pool

and prompts enter in chunks, next to the requests that decode.  The products
with the weights are torch's.  Needs a GPU and the built library.
"""

from __future__ import annotations

import dataclasses
import sys
from typing import List, Optional, Sequence

import torch
import torch.nn.functional as F

from paged_kv_gb300 import pkv


@dataclasses.dataclass
class Config:
    vocab: int = 512
    layers: int = 2
    width: int = 256
    q_heads: int = 8
    kv_heads: int = 2
    head_dim: int = 64
    window: int = 0          # attention window of every second layer; 0: none
    max_pos: int = 4096
    dtype: torch.dtype = torch.bfloat16


class Model:
    """Random weights of a small pre-norm decoder with tied embeddings."""

    def __init__(self, cfg: Config, seed: int = 0, device="cuda"):
        g = torch.Generator().manual_seed(seed)

        def weight(*shape):
            return (torch.randn(shape, generator=g) * shape[-1] ** -0.5).to(cfg.dtype).to(device)

        self.cfg = cfg
        heads = cfg.q_heads + 2 * cfg.kv_heads
        self.embed = weight(cfg.vocab, cfg.width)
        self.layers = [dict(qkv=weight(heads * cfg.head_dim, cfg.width),
                            out=weight(cfg.width, cfg.q_heads * cfg.head_dim),
                            up=weight(4 * cfg.width, cfg.width),
                            down=weight(cfg.width, 4 * cfg.width)) for _ in range(cfg.layers)]
        half = cfg.head_dim // 2
        angle = torch.arange(cfg.max_pos, dtype=torch.float64)[:, None] * (
            10000.0 ** (-torch.arange(half, dtype=torch.float64) / half))
        self.cos_sin = torch.cat([angle.cos(), angle.sin()], 1).float().to(device)

    def norm(self, x):
        return F.rms_norm(x, (self.cfg.width,), eps=1e-5)

    def window(self, layer: int) -> int:
        return self.cfg.window if layer % 2 else 0


@dataclasses.dataclass
class Request:
    prompt: List[int]
    new_tokens: int = 16
    temperature: float = 0.0
    repetition: float = 1.0
    presence: float = 0.0
    frequency: float = 0.0
    bias: Sequence = ()                 # (token, value) pairs
    allowed: Optional[Sequence] = None  # the tokens a grammar allows; None: all


class Engine:
    """Requests of fixed rows, each with its lengths; ``step`` runs one forward pass."""

    def __init__(self, model: Model, requests: Sequence[Request], page_size: int = 16,
                 chunk: int = 64, seed: int = 1, device="cuda"):
        c, n = model.cfg, len(requests)
        self.model, self.requests, self.page_size, self.chunk = model, list(requests), page_size, chunk
        self.seed, self.steps, self.device = seed, 0, torch.device(device)
        self.goal = [len(r.prompt) + r.new_tokens for r in requests]
        if min(len(r.prompt) for r in requests) < 1 or max(self.goal) > c.max_pos:
            raise ValueError("a prompt needs at least one token, and all of a request's "
                             f"tokens at most {c.max_pos} positions")
        width = -(-max(self.goal) // page_size) * page_size
        pages = sum(-(-g // page_size) for g in self.goal)
        self.cached = [0] * n  # positions in the cache
        self.known = [len(r.prompt) for r in requests]  # tokens in the pool
        pool = torch.zeros(n, width, dtype=torch.int32)
        for i, r in enumerate(requests):
            pool[i, :len(r.prompt)] = torch.tensor(r.prompt, dtype=torch.int32)
        self.token_pool = pool.to(device)
        self.page_table = torch.zeros(n, width, dtype=torch.int32, device=device)
        self.free_slots = torch.arange(pages, dtype=torch.int32, device=device) * page_size
        self.used = 0  # of free_slots
        self.caches = [pkv.KVCache.empty(pages, page_size, c.kv_heads, c.head_dim, device)
                       for _ in range(c.layers)]
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def _ints(self, x, dtype=torch.int32):
        return torch.tensor(x, dtype=dtype, device=self.device)

    def _floats(self, x):
        return torch.tensor(x, dtype=torch.float32, device=self.device)

    def forward(self, x, table, cached, device_len, positions, out_loc, longest):
        """The layers on the packed tokens' embeddings."""
        m, c = self.model, self.model.cfg
        for i, (w, cache) in enumerate(zip(m.layers, self.caches)):
            qkv = (m.norm(x) @ w["qkv"].t()).view(x.shape[0], -1, c.head_dim)
            q, k, v = qkv.split([c.q_heads, c.kv_heads, c.kv_heads], 1)
            q = pkv.append_kv(cache, k, v, positions, out_loc, m.cos_sin, q=q, status=self.status)
            o = pkv.paged_attention(q, cache, cached, device_len, table, self.page_table, longest,
                                    window=m.window(i), status=self.status)
            x = x + o.flatten(1) @ w["out"].t()
            x = x + F.silu(m.norm(x) @ w["up"].t()) @ w["down"].t()
        return x

    def adjust(self, logits, rows, device_len):
        """The requests' penalties, biases and grammars, in place."""
        rs = [self.requests[i] for i in rows]
        pairs = [list(r.bias) for r in rs]
        ptr = torch.tensor([0] + [len(p) for p in pairs]).cumsum(0).tolist()
        flat = [p for row in pairs for p in row]
        mask = None
        if any(r.allowed is not None for r in rs):
            words = -(-logits.shape[1] // 32)
            bits = torch.ones(len(rs), words * 32, dtype=torch.int64)
            for i, r in enumerate(rs):
                if r.allowed is not None:
                    bits[i] = 0
                    bits[i, list(r.allowed)] = 1
            mask = (bits.view(len(rs), words, 32) << torch.arange(32)).sum(2)
            mask = torch.where(mask >= 1 << 31, mask - (1 << 32), mask).to(torch.int32)
            mask = mask.to(self.device)
        pkv.adjust_logits(
            logits, token_pool=self.token_pool, table_idx=self._ints(rows),
            prompt_len=self._ints([len(r.prompt) for r in rs]), device_len=device_len,
            repetition=self._floats([r.repetition for r in rs]),
            presence=self._floats([r.presence for r in rs]),
            frequency=self._floats([r.frequency for r in rs]),
            bias_ptr=self._ints(ptr) if flat else None,
            bias_ids=self._ints([t for t, _ in flat]) if flat else None,
            bias_values=self._floats([x for _, x in flat]) if flat else None,
            mask=mask, status=self.status)

    def step(self):
        """One pass over the requests that are not done.  Returns (rows, logits,
        tokens) of those that it sampled (logits as the sampler saw them), or None
        when all are done."""
        rows = [i for i in range(len(self.requests)) if self.known[i] < self.goal[i]]
        if not rows:
            return None
        begin = [self.cached[i] for i in rows]
        end = [min(self.known[i], self.cached[i] + self.chunk) for i in rows]
        n = sum(e - b for b, e in zip(begin, end))
        table, cached, device_len = self._ints(rows), self._ints(begin), self._ints(end)
        free = self.free_slots[self.used:]
        self.used += pkv.alloc_pages(begin, end, self.page_size, free.numel())["total"]
        positions, ids, out_loc, _, _ = pkv.prepare_step(
            cached, device_len, table, self.page_size, free, self.page_table, self.token_pool, n,
            status=self.status)
        x = self.forward(self.model.embed[ids.long()], table, cached, device_len, positions,
                         out_loc, max(e - b for b, e in zip(begin, end)))
        for i, e in zip(rows, end):
            self.cached[i] = e

        # The rows whose last known token has been seen get the next one.
        last, sampled, at = [], [], 0
        for i, b, e in zip(rows, begin, end):
            at += e - b
            if e == self.known[i]:
                last.append(at - 1)
                sampled.append(i)
        self.steps += 1
        if not sampled:
            return [], None, None
        logits = (self.model.norm(x[self._ints(last, torch.int64)]) @ self.model.embed.t()).float()
        lengths = [self.known[i] for i in sampled]
        self.adjust(logits, sampled, self._ints(lengths))
        tokens = pkv.sample_batch(
            logits, self._floats([self.requests[i].temperature for i in sampled]),
            uniform=pkv.philox_uniforms(self.seed, self.steps, len(sampled), device=self.device),
            token_pool=self.token_pool, wb_rows=self._ints(sampled),
            wb_cols=self._ints(lengths, torch.int64), status=self.status)
        for i in sampled:
            self.known[i] += 1
        return sampled, logits, tokens

    def run(self) -> List[List[int]]:
        """Steps until all are done; returns each request's new tokens."""
        while self.step() is not None:
            pass
        status = int(self.status.item())
        if status:
            raise pkv.PkvError(status, f"status word {status:#x}")
        pool = self.token_pool.cpu()
        return [pool[i, len(r.prompt):g].tolist()
                for i, (r, g) in enumerate(zip(self.requests, self.goal))]


def main(argv=None) -> None:
    argv = sys.argv[1:] if argv is None else argv
    n = int(argv[0]) if argv else 8
    new = int(argv[1]) if len(argv) > 1 else 16
    cfg = Config(window=48)
    g = torch.Generator().manual_seed(7)
    requests = []
    for i in range(n):
        length = int(torch.randint(1, 200, (1,), generator=g))
        prompt = torch.randint(0, cfg.vocab, (length,), generator=g).tolist()
        requests.append(Request(prompt, new, temperature=0.8 * (i % 2), repetition=1.1,
                                frequency=0.2, allowed=range(0, cfg.vocab, 2) if i % 3 == 2 else None))
    for i, tokens in enumerate(Engine(Model(cfg), requests).run()[:4]):
        print(f"request {i} ({len(requests[i].prompt)} prompt tokens):", *tokens)


if __name__ == "__main__":
    main()
