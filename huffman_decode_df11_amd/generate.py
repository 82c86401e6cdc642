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

With cache_bits=4 prompt and own positions lie in one paged cache of 4-bit
codes for each layer (quantized_write, quantized_attention), whose pages of
the prompt are the batch's in common; the bounded caches are cut out of what it
holds (quantized_read).  Wishes for the next tokens (penalties, a bias, the
tokens that a grammar allows) are put on the logits of both models
(adjust_logits) before their probabilities are taken.

    python -m huffman_decode_df11_amd.generate --batch 8 --prompt 2000 --new 64
"""
from __future__ import annotations

import argparse
import math
from dataclasses import dataclass
from typing import Dict, List, Optional

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


@dataclass
class Wishes:
    """What a batch's next tokens should be like.  repetition divides the
    logits of tokens that a sequence holds, its prompt's among them (multiplies
    them where negative); presence and frequency are taken off the logits of
    those that were generated, once and for each time; bias is added to a
    token's logit; tokens that allowed [vocab] (bool) leaves out never come."""
    repetition: float = 1.0
    presence: float = 0.0
    frequency: float = 0.0
    bias: Optional[Dict[int, float]] = None
    allowed: Optional[torch.Tensor] = None

    def arguments(self, batch: int, vocab: int, device):
        """Those of adjust_logits that stay the same from call to call."""
        full = lambda x: torch.full((batch,), float(x), device=device)
        a = dict(repetition=full(self.repetition), presence=full(self.presence), frequency=full(self.frequency))
        if not self.repetition > 0.0:
            raise ValueError("repetition must be positive")
        if self.bias:
            if not all(0 <= token < vocab for token in self.bias):
                raise ValueError("a bias is for a token of the vocabulary")
            row = lambda x, dtype: torch.tensor([list(x)], dtype=dtype, device=device).expand(batch, -1).contiguous()
            a["bias"] = row(self.bias.keys(), torch.int64), row(self.bias.values(), torch.float32)
        if self.allowed is not None:
            if self.allowed.shape != (vocab,) or self.allowed.dtype != torch.bool or not self.allowed.any():
                raise ValueError("allowed must say yes or no to each token of the vocabulary, and yes to one")
            bits = torch.zeros(-(-vocab // 32) * 32, dtype=torch.int64)
            bits[:vocab] = self.allowed.cpu()
            words = (bits.view(-1, 32) << torch.arange(32)).sum(1)
            a["mask"] = torch.where(words < 2 ** 31, words, words - 2 ** 32).to(torch.int32).to(device)   # as int32 has the bits
        return a


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

    def probs(self, hidden, temperature: float, adjust=None):
        """Probabilities of the next token, float32 (temperature 0: all of it
        on the likeliest); adjust(logits) may change the logits first."""
        logits = self.head(hidden).float()
        if adjust is not None:
            logits = adjust(logits)
        if temperature == 0.0:
            return torch.zeros_like(logits).scatter_(-1, logits.argmax(-1, keepdim=True), 1.0)
        return torch.softmax(logits / temperature, -1)


class Generator:
    """A batch that continues one prompt.  budget, recent: the bounded
    cache's slots and the latest positions it always keeps; drafts: tokens
    proposed at a time (0: none, one token a round); room: positions a sequence may add; page: positions
    of a page of its own cache.  cache_bits: 16, or 4 for prompt and own
    positions in 4-bit codes (page a multiple of 16 then); wishes: what the
    next tokens should be like."""

    CHUNK = 256    # prompt tokens at a time
    WINDOW = 32    # last prompt tokens, whose attention says what the bounded cache keeps

    def __init__(self, model: Decoder, prompt, batch: int, budget: int = 256, recent: int = 32, drafts: int = 4,
                 room: int = 512, page: int = 16, temperature: float = 1.0, seed: int = 0, cache_bits: int = 16,
                 wishes: Optional[Wishes] = None):
        c, device = model.config, model.device
        if not prompt.numel():
            raise ValueError("the prompt needs a token")
        if cache_bits not in (16, 4):
            raise ValueError("cache_bits must be 16 or 4")
        if cache_bits == 4 and page % 16:
            raise ValueError("pages of 4-bit codes hold a multiple of 16 positions")
        self.model, self.batch, self.recent, self.drafts, self.temperature = model, batch, recent, drafts, temperature
        self.random = torch.Generator(device=device).manual_seed(seed)
        pages = -(-(room + drafts + 1) // page)
        self.room, self.page, self.quantized = room, page, cache_bits == 4
        # prompt: all but its last token, which the sequences' own positions begin with
        if self.quantized:
            self._prefill_quantized(prompt[:-1], budget)
        else:
            self.prefix = self._prefill(prompt[:-1], budget)
            order = torch.randperm(batch * pages, device=device).to(torch.int32)
            self.table = order.view(batch, pages).contiguous()
            self.own = [torch.zeros((2, batch * pages, page, c.kv_heads, c.dim), dtype=torch.bfloat16, device=device)
                        for _ in model.layers]
        self.wishes = None
        if wishes is not None:
            self.wishes = wishes.arguments(batch, c.vocab, device)
            self.prompt_lengths = torch.full((batch,), prompt.numel(), dtype=torch.int32, device=device)
            # the tokens that a sequence holds, and a round's behind them until it is known which of them stay
            self.history = torch.full((batch, prompt.numel() + room + drafts + 1), -1, dtype=torch.int64, device=device)
            self.history[:, :prompt.numel()] = prompt.to(device)
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
        self._bound(P, window, lambda i: (kv[i][0][None], kv[i][1][None]), budget)
        return kv

    def _prefill_quantized(self, prompt, budget: int):
        """The same in a cache of 4-bit codes for each layer: the prompt's whole
        pages the batch's in common, each sequence's own pages behind them,
        which begin with the prompt's last ones."""
        c, model, page = self.model.config, self.model, self.page
        P = prompt.numel()
        shared, own = P // page, -(-(P % page + self.room + self.drafts + 1) // page)
        order = torch.randperm(shared + self.batch * own, device=model.device).to(torch.int32)
        self.table = torch.cat([order[:shared].expand(self.batch, shared), order[shared:].view(self.batch, own)], 1).contiguous()
        self.held = [serve.QuantizedCache.empty(order.numel(), c.kv_heads, page, c.dim, device=model.device) for _ in model.layers]
        window = [None] * c.layers
        first = self.table[:1]   # the prompt in the first sequence's pages
        for at in range(0, P, self.CHUNK):
            n = min(self.CHUNK, P - at)
            position = torch.tensor([at], dtype=torch.int32, device=model.device)

            def attend(i, q, k, v):
                window[i] = q if window[i] is None else torch.cat([window[i], q], 1)[:, -self.WINDOW:]
                return self._attend_quantized(i, q, k, v, position, first)

            model(prompt[None, at:at + n].to(model.device), torch.arange(at, at + n, device=model.device)[None], attend)
        if P % page:   # the positions behind the whole pages, for every sequence
            begun = self.table[:, shared].long()
            for cache in self.held:
                for x in (cache.k_codes, cache.v_codes, cache.k_scales, cache.v_scales):
                    x[begun[1:]] = x[begun[:1]]
        length = torch.tensor([P], dtype=torch.int32, device=model.device)
        self._bound(P, window, lambda i: serve.quantized_read(self.held[i], length, P, block_table=first), budget)

    def _attend_quantized(self, layer, q, k, v, positions, table):
        """New rows at positions [B] on, and attention over them and all before them."""
        cache = self.held[layer]
        lengths = serve.quantized_write(cache, k, v, positions, block_table=table)
        return serve.quantized_attention(q, cache, lengths, block_table=table)

    def _bound(self, P: int, window, rows, budget: int):
        """The bounded caches: what the last prompt tokens' queries, window, give
        the most weight of the P rows of each layer, rows(i) = k, v [1, P, H, D]."""
        c, model = self.model.config, self.model
        self.caches: List[serve.BoundedCache] = []
        for i in range(c.layers):
            if not P:   # a prompt of one token: nothing to keep yet
                self.caches.append(serve.BoundedCache.empty(self.batch, c.kv_heads, budget, c.dim, device=model.device))
                continue
            q = window[i][:, -self.WINDOW:]
            place = torch.arange(P, dtype=torch.int32, device=model.device).expand(1, c.kv_heads, P).contiguous()
            k, v = rows(i)
            whole = serve.BoundedCache(k.transpose(1, 2), v.transpose(1, 2),
                                       torch.zeros((1, c.kv_heads, P), device=model.device), place,
                                       torch.full((1,), P, dtype=torch.int32, device=model.device))
            first = torch.full((1,), P - q.shape[1], dtype=torch.int32, device=model.device)
            serve.cache_attention(q, whole, first)
            cut, _ = serve.cache_compact(whole, torch.full_like(first, P), budget, min(self.recent, budget))
            self.caches.append(serve.BoundedCache(*(t.repeat_interleave(self.batch, 0) for t in (
                cut.k, cut.v, cut.weights, cut.positions, cut.lengths))))

    # ------------------------------------------------------------ one round
    def _positions(self):
        return self.start + self.own_count

    def _adjust(self, ahead: int, drafts=None):
        """What probs() does to logits [B, V] with `ahead` drafts in the history,
        or [B, T, V] with drafts [B, T - 1] behind it; None without wishes."""
        if self.wishes is None:
            return None
        lengths = (self.start + 1 + self.own_count + ahead).to(torch.int32)

        def adjust(logits):
            wishes = dict(self.wishes)
            if "mask" in wishes:
                wishes["mask"] = wishes["mask"].expand(*logits.shape[:-1], -1)   # read with strides of 0
            return serve.adjust_logits(logits, self.history, lengths, prompt_lengths=self.prompt_lengths, drafts=drafts,
                                       out=logits, **wishes)

        return adjust

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
            p = self.model.probs(hidden[:, 0], self.temperature, self._adjust(g))
            ids = torch.multinomial(p, 1, generator=self.random)[:, 0]
            tokens.append(ids)
            probs.append(p)
            if self.wishes is not None:
                self.history.scatter_(1, (self.start + 1 + self.own_count + g).long()[:, None], ids[:, None])
            at = at + 1
        return torch.stack(tokens, 1), torch.stack(probs, 1)

    def score(self, ids):
        """The target's distributions behind each of ids [B, T], the last T of
        the sequences' own positions."""
        T = ids.shape[1]
        own = self.own_count[:, None].long() + torch.arange(T, device=ids.device)
        adjust = self._adjust(0, ids[:, 1:].long().contiguous() if T > 1 else None)
        if self.quantized:
            first = self._positions().to(torch.int32)
            attend = lambda i, q, k, v: self._attend_quantized(i, q, k, v, first, self.table)
            return self.model.probs(self.model(ids, self.start + own, attend), self.temperature, adjust)
        rows = torch.gather(self.table.long(), 1, own // self.page)
        lengths = (self.own_count + T).to(torch.int32)

        def attend(i, q, k, v):
            self.own[i][0, rows, own % self.page], self.own[i][1, rows, own % self.page] = k, v
            return serve.prefix_attention(q, self.prefix[i][0], self.prefix[i][1], self.own[i][0], self.own[i][1], lengths,
                                          block_table=self.table)

        return self.model.probs(self.model(ids, self.start + own, attend), self.temperature, adjust)

    def round(self):
        """Tokens that every sequence gains [B, drafts + 1], -1 behind them, and how many drafts were taken [B].
        Raises ValueError, before anything is done, where a sequence has no room for all of them."""
        if int(self.own_count.max()) + self.drafts + 1 > self.room:
            raise ValueError("the sequences' own positions are full: more room is needed")
        drafts, q = self.draft()
        p = self.score(torch.cat([self.last[:, None], drafts], 1))
        uniforms = torch.rand((self.batch, self.drafts + 1), generator=self.random, device=p.device)
        tokens, taken = serve.verify_drafts(drafts, p, uniforms, q)
        if self.wishes is not None:
            behind = self.start + 1 + self.own_count[:, None].long() + torch.arange(self.drafts + 1, device=p.device)
            self.history.scatter_(1, behind, tokens.long())
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
    ap.add_argument("--cache-bits", type=int, default=16, choices=(16, 4), help="bits of the prompt's and the sequences' positions")
    ap.add_argument("--repetition", type=float, default=1.0, help="divides the logits of tokens that a sequence holds")
    ap.add_argument("--presence", type=float, default=0.0, help="taken off the logits of generated tokens")
    ap.add_argument("--frequency", type=float, default=0.0, help="taken off them for each time that they came")
    a = ap.parse_args()
    model = Decoder(Config())
    prompt = torch.randint(model.config.vocab, (a.prompt,), generator=torch.Generator().manual_seed(1))
    wishes = Wishes(a.repetition, a.presence, a.frequency)
    wishes = wishes if wishes != Wishes() else None
    # a sequence may gain all of a round's tokens in each round in which the slowest gains one
    g = Generator(model, prompt, a.batch, budget=a.budget, drafts=a.drafts, room=(a.new + 1) * (a.drafts + 1),
                  temperature=a.temperature, cache_bits=a.cache_bits, wishes=wishes)
    out, taken = g.generate(a.new)
    print("%d sequences of %d new tokens; %.2f of %d drafts taken in a round" % (len(out), a.new, taken, a.drafts))
    print("first:", out[0][:16])


if __name__ == "__main__":
    main()
