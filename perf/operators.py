"""Cases of the token-generation operators, their plain forms and their 64-bit values.

The operators are those of a generation step around the compressed weights:

* ``prefix_attention``  attention of a batch whose sequences share one long prefix,
* ``cache_attention``   attention over a bounded cache that adds up each slot's weight,
* ``cache_insert``      one token into a bounded cache, evicting the slot of least weight,
* ``cache_compact``     a long cache cut down to its heaviest and latest positions,
* ``verify_drafts``     drafted tokens against the target's probabilities.

``run`` computes them from elementary torch operations, or, with ``own`` set,
through ``huffman_decode_df11_amd.serve``.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
INF = float("inf")
NO_TOKEN = 2 ** 31 - 1   # the position of a slot that holds none


# ------------------------------------------------------------------- the cases
def _prefix(batch, tokens, prefix, suffix, page, heads, kv_heads, dim, dtype, **name):
    return {**name, "op": "prefix_attention", "batch": batch, "tokens": tokens, "prefix": prefix,
            "suffix": suffix, "page": page, "heads": heads, "kv_heads": kv_heads, "dim": dim, "dtype": dtype}


def _attend(batch, tokens, slots, heads, kv_heads, dim, dtype, **name):
    return {**name, "op": "cache_attention", "batch": batch, "tokens": tokens, "slots": slots,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "dtype": dtype}


def _insert(batch, slots, recent, kv_heads, dim, dtype, **name):
    return {**name, "op": "cache_insert", "batch": batch, "slots": slots, "recent": recent,
            "kv_heads": kv_heads, "dim": dim, "dtype": dtype}


def _compact(batch, slots, budget, recent, kv_heads, dim, dtype, **name):
    return {**name, "op": "cache_compact", "batch": batch, "slots": slots, "budget": budget,
            "recent": recent, "kv_heads": kv_heads, "dim": dim, "dtype": dtype}


def _verify(batch, drafts, vocab, dtype, **name):
    return {**name, "op": "verify_drafts", "batch": batch, "drafts": drafts, "vocab": vocab, "dtype": dtype}


def listed():
    return [
        # two requests just behind a short system prompt: a call that is all latency
        _prefix(2, 1, 511, 33, 0, 32, 8, 128, "bf16", name="prefix, 2 requests"),
        # a served batch verifying four drafted tokens behind a document, own positions in pages of 16
        _prefix(24, 5, 8191, 700, 16, 32, 8, 128, "fp16", name="prefix, 24 x 5 drafts, paged"),
        # many requests about one long document, the 8B layer's heads
        _prefix(128, 1, 32768, 1024, 16, 32, 8, 128, "bf16", name="prefix, 128 requests, long"),
        # one request generating from a small bounded cache
        _attend(1, 1, 1024, 32, 8, 128, "bf16", name="cache attention, 1 request"),
        # a served batch, every head its own keys and values of 64
        _attend(33, 1, 4099, 16, 16, 64, "fp16", name="cache attention, 33 requests"),
        # the last tokens of a prompt over the whole prompt: the weights that choose what stays
        _attend(4, 32, 16384, 32, 8, 128, "bf16", name="cache attention, window of 32"),
        # one token into one request's cache
        _insert(1, 500, 64, 8, 128, "bf16", name="insert, 1 request"),
        # one token of a served batch into caches of 4096
        _insert(128, 4096, 256, 8, 128, "bf16", name="insert, 128 requests"),
        # a prompt of a few thousand tokens cut down after its prefill
        _compact(2, 3001, 1000, 100, 8, 128, "fp16", name="compact, 2 prompts"),
        # long prompts of a served batch
        _compact(16, 32768, 4096, 512, 8, 128, "bf16", name="compact, 16 long prompts"),
        # one request with four drafted tokens, the 8B model's vocabulary
        _verify(1, 4, 128256, "fp32", name="verify, 1 request"),
        # a served batch with seven drafted tokens each
        _verify(128, 7, 128256, "bf16", name="verify, 128 requests"),
    ]


def _log(rng, lo, hi):
    """A whole number spread over the logarithm of lo..hi."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("prefix", "prefix", "attend", "attend", "insert", "compact", "verify"))
    dtype = rng.choice(("bf16", "fp16"))
    kv_heads, group, dim = rng.choice(((8, 4, 128), (8, 4, 128), (16, 1, 64), (8, 8, 128), (2, 7, 128), (4, 3, 96),
                                       (4, 2, 256), (5, 5, 64), (1, 8, 80)))
    heads = kv_heads * group
    if op == "prefix":
        tokens = rng.choice((1, 1, rng.randint(2, 8)))
        prefix, suffix = _log(rng, 64, 32768), max(tokens, _log(rng, 8, 1024))
        most = max(1, int(128 * 32 * 128 * 32768 / (heads * dim * tokens * max(prefix, 4096) * 1.1)))
        return _prefix(_log(rng, 1, min(128, most)), tokens, prefix, suffix, rng.choice((0, 16, 16, 64, 7)), heads,
                       kv_heads, dim, dtype)
    if op == "attend":
        tokens = rng.choice((1, 1, rng.randint(2, 32)))
        slots = max(tokens, _log(rng, 16, 16384))
        most = max(1, int(4 * 32 * 16384 * 32 * 128 / (tokens * slots * heads * dim) / 1.1))
        most = min(most, max(1, int(4 * 16384 * 8 * 128 / (slots * kv_heads * dim) / 1.1)))
        return _attend(_log(rng, 1, min(64, most)), tokens, slots, heads, kv_heads, dim, dtype)
    if op == "insert":
        slots = _log(rng, 16, 4096)
        return _insert(_log(rng, 1, 120), slots, rng.randint(1, max(1, slots // 4)), min(8, kv_heads), min(128, dim),
                       dtype)
    if op == "compact":
        slots = _log(rng, 64, 30000)
        budget = max(2, int(slots * rng.uniform(0.06, 0.5)))
        most = max(1, int(16 * 4096 * 8 * 128 / (budget * kv_heads * dim) / 1.1))
        return _compact(_log(rng, 1, min(16, most)), slots, budget, rng.randint(1, max(1, budget // 2)), kv_heads, dim,
                        dtype)
    return _verify(_log(rng, 1, 64), rng.randint(1, 7), _log(rng, 5000, 128256), rng.choice(("fp32", "bf16", "fp16")))


# ------------------------------------------------------------------ the inputs
def _spread(count, least, most):
    """`count` whole numbers evenly spread over least..most."""
    return [least + (i * (most - least)) // max(1, count - 1) if count > 1 else most for i in range(count)]


def _shuffled(values, gen):
    order = torch.randperm(len(values), generator=gen, device="cuda")
    return torch.tensor(values, dtype=torch.int32, device="cuda")[order]


def _suffix_lengths(case):
    return _spread(case["batch"], case["tokens"], case["suffix"])


def _cache(case, gen, seen_more):
    """A bounded cache in use: keys and values, uneven weights with ties among
    them, positions in the order that evictions leave."""
    B, H, C, D, dtype = case["batch"], case["kv_heads"], case["slots"], case["dim"], DTYPES[case["dtype"]]
    k = torch.randn((B, H, C, D), generator=gen, device="cuda", dtype=torch.float32).to(dtype)
    v = torch.randn((B, H, C, D), generator=gen, device="cuda", dtype=torch.float32).to(dtype)
    weights = torch.exp(2.0 * torch.randn((B, H, C), generator=gen, device="cuda"))
    weights[torch.rand((B, H, C), generator=gen, device="cuda") < 0.05] = 0.0
    if seen_more:
        positions = torch.rand((B, H, C + seen_more), generator=gen, device="cuda").argsort(-1)[..., :C]
    else:
        positions = torch.arange(C, device="cuda").expand(B, H, C)
    return {"k": k, "v": v, "weights": weights.contiguous(), "positions": positions.to(torch.int32).contiguous()}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(1000003 * seed + 17)

    def normal(*shape, scale=1.0, dtype=None):
        x = scale * torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32)
        return x.to(dtype or DTYPES[case["dtype"]])

    state = {"case": case}
    op, B = case["op"], case["batch"]
    if op == "prefix_attention":
        T, H, D, page = case["tokens"], case["kv_heads"], case["dim"], case["page"]
        state["q"] = normal(B, T, case["heads"], D, scale=1.5)
        state["prefix_k"], state["prefix_v"] = normal(case["prefix"], H, D), normal(case["prefix"], H, D)
        state["lengths"] = _shuffled(_suffix_lengths(case), gen)
        state["block_table"] = None
        if page:
            per = -(-case["suffix"] // page)
            state["k"], state["v"] = normal(B * per, page, H, D), normal(B * per, page, H, D)
            order = torch.randperm(B * per, generator=gen, device="cuda").to(torch.int32)
            state["block_table"] = order.view(B, per).contiguous()
        else:
            state["k"], state["v"] = normal(B, case["suffix"], H, D), normal(B, case["suffix"], H, D)
    elif op == "cache_attention":
        T, C = case["tokens"], case["slots"]
        state.update(_cache(case, gen, seen_more=C // 2 if T == 1 else 0))
        state["q"] = normal(B, T, case["heads"], case["dim"], scale=1.5)
        if T == 1:   # generation: caches filled to different heights, evictions behind them
            state["lengths"] = _shuffled(_spread(B, max(1, C // 2), C), gen)
            state["pos"] = torch.full((B,), C + C // 2, dtype=torch.int32, device="cuda")
        else:        # the last tokens of a prompt that fills the cache
            state["lengths"] = torch.full((B,), C, dtype=torch.int32, device="cuda")
            state["pos"] = torch.full((B,), C - T, dtype=torch.int32, device="cuda")
    elif op == "cache_insert":
        C = case["slots"]
        state.update(_cache(case, gen, seen_more=C // 2))
        state["k_new"], state["v_new"] = normal(B, case["kv_heads"], case["dim"]), normal(B, case["kv_heads"], case["dim"])
        state["lengths"] = torch.full((B,), C, dtype=torch.int32, device="cuda")
        state["pos"] = torch.full((B,), C + C // 2, dtype=torch.int32, device="cuda")
    elif op == "cache_compact":
        C = case["slots"]
        state.update(_cache(case, gen, seen_more=0))
        state["lengths"] = _shuffled(_spread(B, max(case["budget"], C - C // 4), C), gen)
        state["pos"] = state["lengths"].clone()
    else:
        G, V, dtype = case["drafts"], case["vocab"], DTYPES[case["dtype"]]
        logits = normal(B, G + 1, V, scale=2.0, dtype=torch.float32)
        state["target_probs"] = torch.softmax(logits, -1).to(dtype)
        logits = logits[:, :G] + normal(B, G, V, scale=0.3, dtype=torch.float32)
        draft = torch.softmax(logits, -1)
        race = torch.empty_like(draft).exponential_(generator=gen)
        state["draft_tokens"] = (draft / race).argmax(-1).to(torch.int32)
        state["draft_probs"] = draft.to(dtype)
        state["uniforms"] = torch.rand((B, G + 1), generator=gen, device="cuda")
    return state


# --------------------------------------------------------------- the operators
def _softmax_terms(s):
    """exp(s - max), the sum and the maximum over the last axis; a row of -inf
    alone gives zeros, the sum 0 and the maximum 0."""
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == -INF, torch.zeros_like(m), m)
    e = torch.exp(s - m)
    return e, e.sum(-1, keepdim=True), m


def _plain_prefix(q, prefix_k, prefix_v, k, v, lengths, block_table):
    B, T, Hq, D = q.shape
    P, H = prefix_k.shape[:2]
    G = Hq // H
    if block_table is not None:
        k = k[block_table.long()].reshape(B, -1, H, D)
        v = v[block_table.long()].reshape(B, -1, H, D)
    S = k.shape[1]
    qf = q.float().view(B, T, H, G, D)
    sp = torch.matmul(qf.permute(2, 0, 1, 3, 4).reshape(H, B * T * G, D), prefix_k.float().permute(1, 2, 0).contiguous())
    ss = torch.matmul(qf.permute(0, 2, 1, 3, 4).reshape(B, H, T * G, D), k.float().permute(0, 2, 3, 1).contiguous())
    t = torch.arange(T, device=q.device).repeat_interleave(G)
    seen = lengths.view(B, 1, 1, 1) - (T - 1) + t.view(1, 1, T * G, 1)
    ss = torch.where(torch.arange(S, device=q.device) < seen, ss, -INF)
    s = torch.cat([sp.view(H, B, T * G, P).transpose(0, 1), ss], -1) * (1.0 / math.sqrt(D))
    e, total, m = _softmax_terms(s)
    op = torch.matmul(e[..., :P].transpose(0, 1).reshape(H, B * T * G, P), prefix_v.float().transpose(0, 1).contiguous())
    o = op.view(H, B, T * G, D).transpose(0, 1) + torch.matmul(e[..., P:], v.float().transpose(1, 2).contiguous())
    o = torch.where(total > 0, o / total, 0.0).view(B, H, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D)
    lse = (m + torch.log(total)).view(B, H, T, G).permute(0, 2, 1, 3).reshape(B, T, Hq)
    return o.to(q.dtype), lse


def _plain_attend(q, k, v, weights, positions, lengths, pos):
    B, T, Hq, D = q.shape
    H, C = k.shape[1:3]
    G = Hq // H
    qf = q.float().view(B, T, H, G, D).transpose(1, 2).reshape(B, H, T * G, D)
    s = torch.matmul(qf, k.float().transpose(2, 3).contiguous()) * (1.0 / math.sqrt(D))
    t = torch.arange(T, device=q.device, dtype=torch.int32).repeat_interleave(G)
    used = torch.arange(C, device=q.device) < lengths.view(B, 1, 1)
    seen = positions.unsqueeze(2) <= (pos.view(B, 1) + t).view(B, 1, T * G, 1)
    s = torch.where(used.unsqueeze(2) & seen, s, -INF)
    e, total, _ = _softmax_terms(s)
    p = torch.where(total > 0, e / total, 0.0)
    o = torch.matmul(p, torch.where(used.unsqueeze(3), v.float(), 0.0))
    weights += p.sum(2)
    return o.view(B, H, T, G, D).transpose(1, 2).reshape(B, T, Hq, D).to(q.dtype), weights


def _lowest(key, where):
    """The lowest index at which `key` has its least value among `where`, and
    whether there is one."""
    index = torch.arange(key.shape[-1], device=key.device)
    least = torch.where(where, key, INF).amin(-1, keepdim=True)
    at = torch.where(where & (key == least), index, key.shape[-1]).amin(-1)
    return at.clamp(max=key.shape[-1] - 1), where.any(-1)


def _plain_insert(k_new, v_new, k, v, weights, positions, lengths, pos, recent):
    B, H, C, D = k.shape
    p = pos.view(B, 1, 1)
    used = (torch.arange(C, device=k.device) < lengths.view(B, 1, 1)).expand(B, H, C)
    stale, has_stale = _lowest(torch.zeros_like(weights), used & (positions >= p))
    least, has_least = _lowest(weights, used & (positions <= p - recent))
    oldest, _ = _lowest(positions.double(), used)
    n = lengths.view(B, 1).long()
    slot = torch.where(has_least, least, oldest)
    slot = torch.where(has_stale, stale, slot)
    slot = torch.where(n < C, n, slot)
    at = slot.unsqueeze(-1)
    k.scatter_(2, at.unsqueeze(-1).expand(B, H, 1, D), k_new.unsqueeze(2))
    v.scatter_(2, at.unsqueeze(-1).expand(B, H, 1, D), v_new.unsqueeze(2))
    weights.scatter_(2, at, 0.0)
    positions.scatter_(2, at, p.expand(B, H, 1))
    return slot.to(torch.int32), (lengths + 1).clamp(max=C).to(torch.int32), k, v, weights, positions


def _plain_compact(k, v, weights, positions, lengths, pos, budget, recent):
    B, H, C, D = k.shape
    p = pos.view(B, 1, 1)
    live = (torch.arange(C, device=k.device) < lengths.view(B, 1, 1)) & (positions < p)
    key = torch.where(positions >= p - recent, INF, weights)
    key = torch.where(live, key, -INF)
    order = torch.sort(key, dim=-1, descending=True, stable=True)[1][..., :budget]
    order = torch.where(torch.gather(live, 2, order), order, C)
    order = order.sort(-1)[0]
    there = order < C
    at = order.clamp(max=C - 1)
    rows = at.unsqueeze(-1).expand(B, H, budget, D)
    k2 = torch.where(there.unsqueeze(-1), torch.gather(k, 2, rows), 0.0)
    v2 = torch.where(there.unsqueeze(-1), torch.gather(v, 2, rows), 0.0)
    w2 = torch.where(there, torch.gather(weights, 2, at), 0.0)
    p2 = torch.where(there, torch.gather(positions, 2, at), NO_TOKEN)
    kept = torch.where(there, order, -1).to(torch.int32)
    return k2.to(k.dtype), v2.to(v.dtype), w2, p2.to(torch.int32), lengths.clamp(max=budget).to(torch.int32), kept


def _plain_verify(draft_tokens, target_probs, uniforms, draft_probs):
    B, G = draft_tokens.shape
    d = draft_tokens.long().unsqueeze(-1)
    p = torch.gather(target_probs[:, :G], 2, d).squeeze(-1).double()
    q = torch.gather(draft_probs, 2, d).squeeze(-1).double()
    takes = uniforms[:, :G].double() * q < p
    accepted = takes.to(torch.int32).cumprod(1).sum(1)
    rows = torch.arange(B, device=d.device)
    one = float(1 << 40)   # probabilities as whole multiples of 2^-40
    tp = (target_probs[rows, accepted].float().clamp(0, 1) * one).to(torch.int64)
    dp = (draft_probs[rows, accepted.clamp(max=G - 1)].float().clamp(0, 1) * one).to(torch.int64)
    rest = (tp - torch.where((accepted < G).unsqueeze(1), dp, 0)).clamp(min=0)
    rest = torch.where((rest.sum(1) > 0).unsqueeze(1), rest, tp)
    run = rest.cumsum(1)
    total = run[:, -1]
    u = (uniforms[:, G] * float(1 << 24)).to(torch.int64)
    goal = u * (total >> 24) + ((u * (total & 0xFFFFFF)) >> 24)
    last = torch.where(total > 0, (run <= goal.unsqueeze(1)).sum(1), -1)
    j = torch.arange(G + 1, device=d.device)
    padded = torch.cat([draft_tokens, draft_tokens[:, :1]], 1)
    tokens = torch.where(j < accepted.unsqueeze(1), padded.long(), -1)
    tokens = torch.where(j == accepted.unsqueeze(1), last.unsqueeze(1), tokens)
    return tokens.to(draft_tokens.dtype), accepted.to(torch.int32)


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if own:
        from huffman_decode_df11_amd import serve
        if op == "prefix_attention":
            return serve.prefix_attention(s["q"], s["prefix_k"], s["prefix_v"], s["k"], s["v"], s["lengths"],
                                          block_table=s["block_table"], return_lse=True)
        if op == "verify_drafts":
            return serve.verify_drafts(s["draft_tokens"], s["target_probs"], s["uniforms"], s["draft_probs"])
        cache = serve.BoundedCache(s["k"], s["v"], s["weights"], s["positions"], s["lengths"])
        if op == "cache_attention":
            return serve.cache_attention(s["q"], cache, s["pos"]), s["weights"]
        if op == "cache_insert":
            slots, lengths = serve.cache_insert(cache, s["k_new"], s["v_new"], s["pos"], case["recent"])
            return slots, lengths, s["k"], s["v"], s["weights"], s["positions"]
        cut, kept = serve.cache_compact(cache, s["pos"], case["budget"], case["recent"])
        return cut.k, cut.v, cut.weights, cut.positions, cut.lengths, kept
    if op == "prefix_attention":
        return _plain_prefix(s["q"], s["prefix_k"], s["prefix_v"], s["k"], s["v"], s["lengths"], s["block_table"])
    if op == "verify_drafts":
        return _plain_verify(s["draft_tokens"], s["target_probs"], s["uniforms"], s["draft_probs"])
    if op == "cache_attention":
        return _plain_attend(s["q"], s["k"], s["v"], s["weights"], s["positions"], s["lengths"], s["pos"])
    if op == "cache_insert":
        return _plain_insert(s["k_new"], s["v_new"], s["k"], s["v"], s["weights"], s["positions"], s["lengths"],
                             s["pos"], case["recent"])
    return _plain_compact(s["k"], s["v"], s["weights"], s["positions"], s["lengths"], s["pos"], case["budget"],
                          case["recent"])


# -------------------------------------------------------------------- the work
def work(case):
    op, B = case["op"], case["batch"]
    if op == "verify_drafts":
        # one row of the target's probabilities for each request and, where a draft
        # is refused (about a tenth of the tokens drawn here), the drafter's row too
        G, V, size = case["drafts"], case["vocab"], DTYPES[case["dtype"]].itemsize
        refused = 1.0 - 0.9 ** G
        return {"bytes": B * (V * size * (1 + refused) + G * (2 * size + 4 + 4) + 4 + 4 * (G + 2)), "flops": B * V * 3.0}
    H, D, size = case["kv_heads"], case["dim"], 2
    if op == "prefix_attention":
        T, Hq, P = case["tokens"], case["heads"], case["prefix"]
        lengths = _suffix_lengths(case)
        seen = sum(sum(n - (T - 1) + t for t in range(T)) for n in lengths)
        table = sum(-(-n // case["page"]) for n in lengths) * 4 if case["page"] else 0
        read = 2 * (P + sum(lengths)) * H * D * size + B * T * Hq * D * size + B * 4 + table
        return {"bytes": read + B * T * Hq * (D * size + 4), "flops": 4.0 * Hq * D * (B * T * P + seen)}
    C = case["slots"]
    if op == "cache_attention":
        T, Hq = case["tokens"], case["heads"]
        slots = sum(_spread(B, max(1, C // 2), C)) if T == 1 else B * C
        # keys, values, positions, weights in and out; queries and outputs
        moved = slots * H * (2 * D * size + 4 + 8) + 2 * B * T * Hq * D * size + B * 8
        return {"bytes": moved, "flops": 4.0 * Hq * D * T * slots}
    if op == "cache_insert":
        return {"bytes": B * H * (C * 8 + 4 * D * size + 8 + 4) + B * 12, "flops": 2.0 * B * H * C}
    slots = sum(_spread(B, max(case["budget"], C - C // 4), C))
    kept = B * H * case["budget"]
    return {"bytes": slots * H * 8 + kept * (4 * D * size + 8 + 4) + B * 12, "flops": 2.0 * slots * H}


# ------------------------------------------------------- the values in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    op, B = case["op"], case["batch"]
    if op == "prefix_attention":
        q = s["q"].double()
        T, Hq, D = q.shape[1:]
        H = case["kv_heads"]
        group = Hq // H
        out, lse = torch.zeros_like(q), torch.full((B, T, Hq), -INF, dtype=torch.float64, device="cuda")
        for h in range(H):
            pk, pv = s["prefix_k"][:, h].double(), s["prefix_v"][:, h].double()
            for b in range(B):
                n = int(s["lengths"][b])
                if s["block_table"] is None:
                    k, v = s["k"][b, :n, h].double(), s["v"][b, :n, h].double()
                else:
                    pages = s["block_table"][b].long()
                    k = s["k"][pages, :, h].reshape(-1, D)[:n].double()
                    v = s["v"][pages, :, h].reshape(-1, D)[:n].double()
                rows = q[b, :, h * group:(h + 1) * group].reshape(T * group, D)
                sc = rows @ torch.cat([pk, k]).T / D ** 0.5
                for t in range(T - 1):
                    sc[t * group:(t + 1) * group, case["prefix"] + n - (T - 1) + t:] = -INF
                lse[b, :, h * group:(h + 1) * group] = torch.logsumexp(sc, 1).view(T, group)
                out[b, :, h * group:(h + 1) * group] = (torch.softmax(sc, 1) @ torch.cat([pv, v])).view(T, group, D)
        return out, lse
    if op == "cache_attention":
        q, weights = s["q"].double(), s["weights"].double()
        T, Hq, D = q.shape[1:]
        H = case["kv_heads"]
        group = Hq // H
        out = torch.zeros_like(q)
        for b in range(B):
            n = int(s["lengths"][b])
            for h in range(H):
                rows = q[b, :, h * group:(h + 1) * group].reshape(T * group, D)
                sc = rows @ s["k"][b, h, :n].double().T / D ** 0.5
                for t in range(T):
                    sc[t * group:(t + 1) * group, s["positions"][b, h, :n] > s["pos"][b] + t] = -INF
                p = torch.softmax(sc, 1)
                weights[b, h, :n] += p.sum(0)
                out[b, :, h * group:(h + 1) * group] = (p @ s["v"][b, h, :n].double()).view(T, group, D)
        return out, weights
    if op == "cache_insert":
        pos, recent = int(s["pos"][0]), case["recent"]
        slots = torch.zeros((B, case["kv_heads"]), dtype=torch.int32, device="cuda")
        for b in range(B):
            for h in range(case["kv_heads"]):
                w, at = s["weights"][b, h].cpu().numpy(), s["positions"][b, h].cpu().numpy()
                free = np.nonzero(at <= pos - recent)[0]
                i = int(free[np.argmin(w[free])] if len(free) else np.argmin(at))   # the first of equals
                slots[b, h] = i
                s["k"][b, h, i], s["v"][b, h, i] = s["k_new"][b, h], s["v_new"][b, h]
                s["weights"][b, h, i], s["positions"][b, h, i] = 0.0, pos
        return slots, s["lengths"], s["k"].double(), s["v"].double(), s["weights"].double(), s["positions"]
    if op == "cache_compact":
        H, D, budget, recent = case["kv_heads"], case["dim"], case["budget"], case["recent"]
        k = torch.zeros((B, H, budget, D), dtype=torch.float64, device="cuda")
        v, w = torch.zeros_like(k), torch.zeros((B, H, budget), dtype=torch.float64, device="cuda")
        kept = torch.full((B, H, budget), -1, dtype=torch.int32, device="cuda")
        for b in range(B):
            n = int(s["lengths"][b])
            for h in range(H):
                old = s["weights"][b, h, :n].double().cpu().numpy()
                slot = np.arange(n)
                late = slot >= n - recent     # slots are positions here: a prompt's cache, in order
                rank = np.lexsort((slot, np.where(late, 0.0, -old), ~late))   # the last key counts first
                keep = torch.from_numpy(np.sort(rank[:budget])).cuda()
                m = len(keep)
                kept[b, h, :m] = keep
                k[b, h, :m], v[b, h, :m] = s["k"][b, h, keep].double(), s["v"][b, h, keep].double()
                w[b, h, :m] = s["weights"][b, h, keep].double()
        return k, v, w, kept, torch.full((B,), budget, dtype=torch.int32, device="cuda"), kept
    G = case["drafts"]
    tokens = torch.full((B, G + 1), -1, dtype=torch.int32, device="cuda")
    accepted = torch.zeros((B,), dtype=torch.int32, device="cuda")
    for b in range(B):
        n = 0
        while n < G:
            d = int(s["draft_tokens"][b, n])
            p, q = float(s["target_probs"][b, n, d]), float(s["draft_probs"][b, n, d])
            if not float(s["uniforms"][b, n]) * q < p:
                break
            tokens[b, n] = d
            n += 1
        accepted[b] = n
        rest = s["target_probs"][b, n].double()
        if n < G:
            rest = (rest - s["draft_probs"][b, n].double()).clamp(min=0)
        run = rest.cumsum(0)
        u = s["uniforms"][b, G].double() * run[-1]
        tokens[b, n] = int(torch.searchsorted(run, u.view(1), right=True)[0])
    return tokens, accepted
