"""The generation operators in 64 bits on the CPU, from their definitions,
and the error bounds the GPU results are held to."""
import math

import torch

NO_TOKEN = 2 ** 31 - 1
# half a unit in the last place of a value near 1, relative
UNIT = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def attend(q, k, v, scale):
    """One row over its visible keys: output, lse, probabilities and the
    output's error bound.  The bound: the result and each probability are
    rounded to the operands' type (unit u; float16 probabilities below its
    normal range by up to 2^-25 of the largest), and a logit of up to 256
    float32 products and sums of terms of a size near 1, its exponential and
    the sums err by less than 2^-12 relative in all."""
    u = UNIT[q.dtype]
    q, k, v = q.double(), k.double(), v.double()
    if k.shape[0] == 0:
        return torch.zeros(q.shape[0], dtype=torch.float64), -math.inf, torch.zeros(0, dtype=torch.float64), \
            torch.zeros(q.shape[0], dtype=torch.float64)
    s = (k @ q) * scale
    p = torch.softmax(s, 0)
    out = p @ v
    bound = u * out.abs() + (u + 2.0 ** -12) * (p @ v.abs()) + 2.0 ** -24 * p.max() * v.abs().sum(0)
    return out, float(torch.logsumexp(s, 0)), p, bound


def prefix_attention(q, pk, pv, k, v, lengths, table=None, scale=None):
    B, T, Hq, D = q.shape
    P, H = pk.shape[:2]
    G = Hq // H
    scale = D ** -0.5 if scale is None else scale
    out, bound = torch.zeros(B, T, Hq, D, dtype=torch.float64), torch.zeros(B, T, Hq, D, dtype=torch.float64)
    lse = torch.zeros(B, T, Hq, dtype=torch.float64)
    for b in range(B):
        if table is None:
            S = k.shape[1]
            place = [(b, s) for s in range(S)]
        else:
            page = k.shape[1]
            S = table.shape[1] * page
            place = [(int(table[b, s // page]), s % page) for s in range(S)]
        n = max(0, min(int(lengths[b]), S))
        for t in range(T):
            seen = [x for x in place[:max(0, n - T + 1 + t)] if 0 <= x[0] < k.shape[0]]
            for h in range(Hq):
                kk = torch.stack([k[i, j, h // G] for i, j in seen]) if seen else k.new_zeros(0, D)
                vv = torch.stack([v[i, j, h // G] for i, j in seen]) if seen else v.new_zeros(0, D)
                out[b, t, h], lse[b, t, h], _, bound[b, t, h] = attend(
                    q[b, t, h], torch.cat([pk[:, h // G], kk]), torch.cat([pv[:, h // G], vv]), scale)
    return out, lse, bound


def cache_attention(q, k, v, weights, positions, lengths, pos, scale=None):
    B, T, Hq, D = q.shape
    H, C = k.shape[1:3]
    G = Hq // H
    scale = D ** -0.5 if scale is None else scale
    out, bound = torch.zeros(B, T, Hq, D, dtype=torch.float64), torch.zeros(B, T, Hq, D, dtype=torch.float64)
    w = weights.double().clone()
    for b in range(B):
        n = max(0, min(int(lengths[b]), C))
        for t in range(T):
            for h in range(Hq):
                at = positions[b, h // G, :n]
                seen = ((at >= 0) & (at <= int(pos[b]) + t)).nonzero()[:, 0]
                out[b, t, h], _, p, bound[b, t, h] = attend(q[b, t, h], k[b, h // G, seen], v[b, h // G, seen], scale)
                w[b, h // G, seen] += p
    return out, w, bound


def _order(w):
    """A weight's place in the order: NaN below everything."""
    return -math.inf if w != w else w


def cache_insert(positions, weights, lengths, pos, recent):
    """The slots taken and the new lengths."""
    B, H, C = weights.shape
    slots, new = torch.full((B, H), -1, dtype=torch.int32), lengths.clone()
    for b in range(B):
        p, n = int(pos[b]), max(0, min(int(lengths[b]), C))
        new[b] = n
        if p < 0:
            continue
        new[b] = min(n + 1, C)
        for h in range(H):
            at, w = positions[b, h].tolist(), weights[b, h].tolist()
            stale = [i for i in range(n) if at[i] >= p or at[i] < 0]
            free = [i for i in range(n) if 0 <= at[i] <= p - recent]
            if n < C:
                slots[b, h] = n
            elif stale:
                slots[b, h] = stale[0]
            elif free:
                slots[b, h] = min(free, key=lambda i: (0 if w[i] != w[i] else 1, _order(w[i]), i))
            else:
                slots[b, h] = min(range(n), key=lambda i: (at[i], i))
    return slots, new


def cache_compact(positions, weights, lengths, pos, budget, recent):
    """The kept slots [B, H, budget], -1 behind them."""
    B, H, C = weights.shape
    kept = torch.full((B, H, budget), -1, dtype=torch.int32)
    for b in range(B):
        p, n = int(pos[b]), max(0, min(int(lengths[b]), C))
        for h in range(H):
            at, w = positions[b, h].tolist(), weights[b, h].tolist()
            live = [i for i in range(n) if 0 <= at[i] < p]
            late = [i for i in live if at[i] >= p - recent]
            others = sorted((i for i in live if at[i] < p - recent),
                            key=lambda i: (1 if w[i] != w[i] else 0, -_order(w[i]), i))
            keep = sorted((late + others)[:budget])
            kept[b, h, :len(keep)] = torch.tensor(keep, dtype=torch.int32)
    return kept


def _whole(p):
    p = p.double()
    p = torch.where(p > 0, p, 0.0).clamp(max=1.0)
    return [int(x) for x in (p * 2.0 ** 40).floor().tolist()]


def verify_drafts(draft_tokens, target, uniforms, draft=None, counts=None):
    B, G = draft_tokens.shape
    V = target.shape[2]
    tokens, accepted = torch.full((B, G + 1), -1, dtype=draft_tokens.dtype), torch.zeros(B, dtype=torch.int32)
    for b in range(B):
        count = G if counts is None else max(0, min(int(counts[b]), G))
        n = 0
        while n < count:
            d = int(draft_tokens[b, n])
            inside = 0 <= d < V
            p = float(target[b, n, d]) if inside else 0.0
            q = (1.0 if draft is None else float(draft[b, n, d])) if inside else 0.0
            if not float(uniforms[b, n]) * q < p:
                break
            tokens[b, n] = d
            n += 1
        accepted[b] = n
        p = _whole(target[b, n])
        rest = p
        if n < count:
            if draft is None:
                q = [0] * V
                if 0 <= int(draft_tokens[b, n]) < V:
                    q[int(draft_tokens[b, n])] = 1 << 40
            else:
                q = _whole(draft[b, n])
            rest = [max(x - y, 0) for x, y in zip(p, q)]
            if sum(rest) == 0:
                rest = p
        goal = int(float(uniforms[b, G]) * 2 ** 24) * sum(rest) >> 24
        run = 0
        for i, x in enumerate(rest):
            run += x
            if goal < run:
                tokens[b, n] = i
                break
    return tokens, accepted
