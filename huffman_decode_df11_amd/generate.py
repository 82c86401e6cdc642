"""Speculative generation with compressed weights: a small decoder whose
matrices stay DFloat11-compressed on the GPU, run by the generation
operators of serve.py.

[P2] "DFloat11：用于高效 GPU 推理的 LLM 和扩散模型无损压缩" "工作原理": the
     compressed weights serve token generation, each matrix restored right
     before its product.

A batch of sequences continues one prompt.  The model drafts for itself: it
proposes tokens one at a time over a bounded cache (the prompt's heaviest and
latest positions, cache_compact; new tokens in the place of the lightest,
cache_insert; cache_attention), then scores all of a sequence's drafts at
once over the whole prompt, which the batch shares, and the sequence's own
positions in pages (prefix_attention).  verify_drafts takes the drafts that
the full cache would have taken, so what comes out is distributed as without
drafting, whatever the bounded cache has dropped.

    python -m huffman_decode_df11_amd.generate --batch 8 --prompt 2000 --new 64
"""
from __future__ import annotations

import argparse
import math
from dataclasses import dataclass
from typing import List

import torch

from . import nn as dnn
from . import serve


@dataclass
class Config:
    layers: int = 2
    hidden: int = 512
    heads: int = 8
    kv_heads: int = 2
    dim: int = 64
    ffn: int = 1024
    vocab: int = 2048


class Layer:
    def __init__(self, c: Config, weight):
        self.q, self.k, self.v = (weight(n * c.dim, c.hidden) for n in (c.heads, c.kv_heads, c.kv_heads))
        self.o = weight(c.hidden, c.heads * c.dim)
        self.gate, self.up, self.down = weight(c.ffn, c.hidden), weight(c.ffn, c.hidden), weight(c.hidden, c.ffn)


class Decoder:
    """A decoder of random weights, every matrix compressed (DF11Linear,
    DF11Embedding): RMS norm, rotary positions, grouped key heads, gated
    feed-forward."""

    def __init__(self, config: Config, seed: int = 0, device="cuda"):
        self.config, self.device = config, torch.device(device)
        g = torch.Generator().manual_seed(seed)

        def weight(rows, cols):
            w = torch.randn((rows, cols), generator=g) / math.sqrt(cols)
            return dnn.DF11Linear(w.to(torch.bfloat16), device=device, deterministic=True)

        self.embed = dnn.DF11Embedding(torch.randn((config.vocab, config.hidden), generator=g).to(torch.bfloat16),
                                       device=device)
        self.layers = [Layer(config, weight) for _ in range(config.layers)]
        self.head = weight(config.vocab, config.hidden)
        self.inverse = 10000.0 ** (-torch.arange(0, config.dim, 2, device=device, dtype=torch.float32) / config.dim)

    def _norm(self, x):
        return (x.float() * torch.rsqrt(x.float().square().mean(-1, keepdim=True) + 1e-6)).to(x.dtype)

    def _turn(self, x, positions):
        """Rotary positions: x [B, T, H, D], positions [B, T]."""
        angle = positions[..., None, None].float() * self.inverse
        a, b = x.float().chunk(2, -1)
        return torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()], -1).to(x.dtype)

    def __call__(self, ids, positions, attend):
        """The final hidden states of ids [B, T] at positions [B, T];
        attend(layer, q, k, v) is the attention, over whatever cache."""
        c = self.config
        B, T = ids.shape
        x = self.embed(ids)
        for i, layer in enumerate(self.layers):
            h = self._norm(x)
            q = self._turn(layer.q(h).view(B, T, c.heads, c.dim), positions)
            k = self._turn(layer.k(h).view(B, T, c.kv_heads, c.dim), positions)
            v = layer.v(h).view(B, T, c.kv_heads, c.dim)
            x = x + layer.o(attend(i, q, k, v).reshape(B, T, c.heads * c.dim))
            h = self._norm(x)
            x = x + layer.down(torch.nn.functional.silu(layer.gate(h)) * layer.up(h))
        return self._norm(x)

    def probs(self, hidden, temperature: float):
        """Probabilities of the next token, float32 (temperature 0: all of it
        on the likeliest)."""
        logits = self.head(hidden).float()
        if temperature == 0.0:
            return torch.zeros_like(logits).scatter_(-1, logits.argmax(-1, keepdim=True), 1.0)
        return torch.softmax(logits / temperature, -1)


class Generator:
    """A batch that continues one prompt.  budget, recent: the bounded
    cache's slots and the latest positions it always keeps; drafts: tokens
    proposed at a time (0: none, one token a round); room: positions a sequence may add; page: positions
    of a page of its own cache."""

    CHUNK = 256    # prompt tokens at a time
    WINDOW = 32    # last prompt tokens, whose attention says what the bounded cache keeps

    def __init__(self, model: Decoder, prompt, batch: int, budget: int = 256, recent: int = 32, drafts: int = 4,
                 room: int = 512, page: int = 16, temperature: float = 1.0, seed: int = 0):
        c, device = model.config, model.device
        if not prompt.numel():
            raise ValueError("the prompt needs a token")
        self.model, self.batch, self.recent, self.drafts, self.temperature = model, batch, recent, drafts, temperature
        self.random = torch.Generator(device=device).manual_seed(seed)
        pages = -(-(room + drafts + 1) // page)
        self.room, self.page = room, page
        # prompt: all but its last token, which the sequences' own positions begin with
        self.prefix = self._prefill(prompt[:-1], budget)
        order = torch.randperm(batch * pages, device=device).to(torch.int32)
        self.table = order.view(batch, pages).contiguous()
        self.own = [torch.zeros((2, batch * pages, page, c.kv_heads, c.dim), dtype=torch.bfloat16, device=device)
                    for _ in model.layers]
        self.own_count = torch.zeros(batch, dtype=torch.int32, device=device)   # own positions that stay
        self.start = prompt.numel() - 1
        self.last = prompt[-1:].expand(batch).to(device)

    def _prefill(self, prompt, budget: int):
        """The prompt's keys and values for each layer, and the bounded caches
        cut out of them (one for each sequence)."""
        c, model = self.model.config, self.model
        P = prompt.numel()
        kv = [torch.empty((2, P, c.kv_heads, c.dim), dtype=torch.bfloat16, device=model.device) for _ in model.layers]
        window = [None] * c.layers
        for at in range(0, P, self.CHUNK):
            n = min(self.CHUNK, P - at)
            lengths = torch.tensor([n], dtype=torch.int32, device=model.device)

            def attend(i, q, k, v):
                kv[i][0, at:at + n], kv[i][1, at:at + n] = k[0], v[0]
                window[i] = q if window[i] is None else torch.cat([window[i], q], 1)[:, -self.WINDOW:]
                return serve.prefix_attention(q, kv[i][0, :at], kv[i][1, :at], k, v, lengths)

            model(prompt[None, at:at + n].to(model.device), torch.arange(at, at + n, device=model.device)[None], attend)
        self.caches: List[serve.BoundedCache] = []
        for i in range(c.layers):
            if not P:   # a prompt of one token: nothing to keep yet
                self.caches.append(serve.BoundedCache.empty(self.batch, c.kv_heads, budget, c.dim, device=model.device))
                continue
            q = window[i][:, -self.WINDOW:]
            place = torch.arange(P, dtype=torch.int32, device=model.device).expand(1, c.kv_heads, P).contiguous()
            whole = serve.BoundedCache(kv[i][0][None].transpose(1, 2), kv[i][1][None].transpose(1, 2),
                                       torch.zeros((1, c.kv_heads, P), device=model.device), place,
                                       torch.full((1,), P, dtype=torch.int32, device=model.device))
            first = torch.full((1,), P - q.shape[1], dtype=torch.int32, device=model.device)
            serve.cache_attention(q, whole, first)
            cut, _ = serve.cache_compact(whole, torch.full_like(first, P), budget, min(self.recent, budget))
            self.caches.append(serve.BoundedCache(*(t.repeat_interleave(self.batch, 0) for t in (
                cut.k, cut.v, cut.weights, cut.positions, cut.lengths))))
        return kv

    # ------------------------------------------------------------ one round
    def _positions(self):
        return self.start + self.own_count

    def draft(self):
        """Tokens proposed over the bounded caches [B, drafts], and the
        distributions they were drawn from (None without drafts)."""
        if not self.drafts:
            return self.last.new_zeros((self.batch, 0)), None
        tokens, probs, ids, at = [], [], self.last, self._positions()
        for g in range(self.drafts + 1):
            def attend(i, q, k, v):
                cache = self.caches[i]
                _, lengths = serve.cache_insert(cache, k[:, 0], v[:, 0], at, self.recent)
                cache.set_lengths(lengths)
                return serve.cache_attention(q, cache, at)

            hidden = self.model(ids[:, None], at[:, None], attend)
            if g == self.drafts:
                break   # the last draft's key and value are in the cache now, for the round behind it
            p = self.model.probs(hidden[:, 0], self.temperature)
            ids = torch.multinomial(p, 1, generator=self.random)[:, 0]
            tokens.append(ids)
            probs.append(p)
            at = at + 1
        return torch.stack(tokens, 1), torch.stack(probs, 1)

    def score(self, ids):
        """The target's distributions behind each of ids [B, T], the last T of
        the sequences' own positions."""
        T = ids.shape[1]
        own = self.own_count[:, None].long() + torch.arange(T, device=ids.device)
        rows = torch.gather(self.table.long(), 1, own // self.page)
        lengths = (self.own_count + T).to(torch.int32)

        def attend(i, q, k, v):
            self.own[i][0, rows, own % self.page], self.own[i][1, rows, own % self.page] = k, v
            return serve.prefix_attention(q, self.prefix[i][0], self.prefix[i][1], self.own[i][0], self.own[i][1], lengths,
                                          block_table=self.table)

        return self.model.probs(self.model(ids, self.start + own, attend), self.temperature)

    def round(self):
        """Tokens that every sequence gains [B, drafts + 1], -1 behind them, and how many drafts were taken [B]."""
        drafts, q = self.draft()
        p = self.score(torch.cat([self.last[:, None], drafts], 1))
        uniforms = torch.rand((self.batch, self.drafts + 1), generator=self.random, device=p.device)
        tokens, taken = serve.verify_drafts(drafts, p, uniforms, q)
        self.own_count = self.own_count + taken + 1
        for cache in self.caches:
            cache.forget(self._positions())   # the refused drafts, before their positions are taken by others
        self.last = torch.gather(tokens, 1, taken[:, None].long())[:, 0]
        return tokens, taken

    def generate(self, count: int):
        """At least `count` new tokens of every sequence: a list of token lists
        (the caches' room bounds the number of rounds), and the mean number
        of drafts taken in a round."""
        out, taken, rounds = [[] for _ in range(self.batch)], 0.0, 0
        while min(len(s) for s in out) < count:
            if int(self.own_count.max()) + self.drafts + 1 > self.room:
                raise ValueError("the sequences' own positions are full: more room is needed")
            tokens, n = self.round()
            for s, row in zip(out, tokens.tolist()):
                s.extend(t for t in row if t >= 0)
            taken, rounds = taken + float(n.float().mean()), rounds + 1
        return [s[:count] for s in out], taken / max(1, rounds)


def main():
    ap = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    ap.add_argument("--batch", type=int, default=8)
    ap.add_argument("--prompt", type=int, default=2000, help="prompt tokens")
    ap.add_argument("--new", type=int, default=64, help="tokens each sequence gains")
    ap.add_argument("--drafts", type=int, default=4)
    ap.add_argument("--budget", type=int, default=256, help="slots of the bounded caches")
    ap.add_argument("--temperature", type=float, default=1.0)
    a = ap.parse_args()
    model = Decoder(Config())
    prompt = torch.randint(model.config.vocab, (a.prompt,), generator=torch.Generator().manual_seed(1))
    # a sequence may gain all of a round's tokens in each round in which the slowest gains one
    g = Generator(model, prompt, a.batch, budget=a.budget, drafts=a.drafts, room=(a.new + 1) * (a.drafts + 1),
                  temperature=a.temperature)
    out, taken = g.generate(a.new)
    print("%d sequences of %d new tokens; %.2f of %d drafts taken in a round" % (len(out), a.new, taken, a.drafts))
    print("first:", out[0][:16])


if __name__ == "__main__":
    main()
