"""Operators of a generation step around the compressed weights.

[P2] "DFloat11：用于高效 GPU 推理的 LLM 和扩散模型无损压缩" "工作原理": the
     compressed weights serve token generation; what runs between their
     products is here, as HIP kernels in libdf11:

* ``prefix_attention``  attention of sequences that share one prefix, read
  once for all of them (several drafted tokens a sequence at a time too);
* ``BoundedCache`` with ``cache_attention`` (attention that adds up the
  weight each slot gets), ``cache_insert`` (one token in, the slot of least
  weight out) and ``cache_compact`` (a long cache cut down to its heaviest
  and latest slots);
* ``verify_drafts``     drafted tokens against the target's probabilities.

Argument checks and marshalling only; there is no fallback implementation.
Work is enqueued on ``stream`` (the device's current stream when None);
outputs and workspaces are allocated on it.
"""
from __future__ import annotations

import struct
from typing import Optional

import torch

from . import _lib
from ._lib import check, lib

NO_TOKEN = _lib.DF11_NO_TOKEN   # position of a cache slot that holds no token

_DTYPES = {torch.bfloat16: _lib.DF11_BF16, torch.float16: _lib.DF11_FP16}
_PROBS = {**_DTYPES, torch.float32: _lib.DF11_FP32}
# The argument structs of df11.h: every field is 8 bytes wide.
_PREFIX_ARGS = struct.Struct("28qd")
_CACHE = struct.Struct("13q")
_CACHE_ARGS = struct.Struct("8qd")
_VERIFY_ARGS = struct.Struct("16q")


def _refuse(cond: bool, text: str) -> None:
    if cond:
        raise ValueError(text)


def _on(name: str, t, dtype, device, shape=None) -> int:
    """The address of a contiguous tensor of this type, device and shape."""
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    _refuse(t.device != device, "%s is on %s, the other operands on %s" % (name, t.device, device))
    _refuse(shape is not None and tuple(t.shape) != shape, "%s has shape %s, not %s" % (name, tuple(t.shape), shape))
    _refuse(not t.is_contiguous(), "%s must be contiguous" % name)
    return t.data_ptr()


def _rows(name: str, t, like, shape):
    """The strides of a tensor of rows (last axis contiguous) like `like`."""
    if t.dtype != like.dtype:
        raise TypeError("%s must be %s, got %s" % (name, like.dtype, t.dtype))
    _refuse(t.device != like.device, "%s is on %s, the other operands on %s" % (name, t.device, like.device))
    _refuse(tuple(t.shape) != shape, "%s has shape %s, not %s" % (name, tuple(t.shape), shape))
    s = t.stride()
    if 1 in shape:   # the stride of an axis of one is never used
        s = tuple(0 if n == 1 else x for n, x in zip(shape, s))
    _refuse(s[-1] != 1 and shape[-1] > 1, "the last axis of %s must be contiguous" % name)
    return s


def _operand(name: str, t, table=_DTYPES) -> int:
    _refuse(not t.is_cuda, "%s must be on the GPU" % name)
    code = table.get(t.dtype)
    if code is None:
        raise TypeError("%s must be one of %s, got %s" % (name, ", ".join(str(d) for d in table), t.dtype))
    return code


class _Work:
    """The device and stream of a call, for its allocations and launches."""

    def __init__(self, device, stream):
        self.device = device
        self.guard = None
        if device.index != torch.cuda.current_device():
            self.guard = torch.cuda.device(device)
        self.stream = stream

    def __enter__(self):
        if self.guard is not None:
            self.guard.__enter__()
        if self.stream is None:
            self.ctx, self.handle = None, torch.cuda.current_stream().cuda_stream
        else:
            self.ctx, self.handle = torch.cuda.stream(self.stream), self.stream.cuda_stream
            self.ctx.__enter__()
        return self.handle

    def __exit__(self, *exc):
        if self.ctx is not None:
            self.ctx.__exit__(*exc)
        if self.guard is not None:
            self.guard.__exit__(*exc)
        return False


def _workspace(nbytes: int, device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def prefix_attention(q, prefix_k, prefix_v, k, v, lengths, *, block_table=None, scale: Optional[float] = None,
                     out=None, return_lse: bool = False, stream=None):
    """Attention of a batch whose sequences share a prefix.

    q [B, T, Hq, D]: T query tokens for each sequence, the last T of its own
    positions.  prefix_k, prefix_v [P, Hkv, D], shared by all sequences.
    k, v [B, S, Hkv, D]: each sequence's own positions, or, with block_table
    [B, pages] int32, pages [N, page, Hkv, D].  lengths [B] int32: how many
    own positions a sequence has, its query tokens among them (token t sees
    the whole prefix and lengths - T + 1 + t own positions).  bfloat16 or
    float16; Hq a multiple of Hkv; D a multiple of 8 up to 256.  The scale
    is 1 / sqrt(D) when None.  Returns out [B, T, Hq, D], and with
    return_lse also lse [B, T, Hq] float32.  A row that sees no position is
    zero (lse -inf)."""
    code = _operand("q", q)
    _refuse(q.dim() != 4, "q must be [B, T, Hq, D]")
    B, T, Hq, D = q.shape
    _refuse(prefix_k.dim() != 3 or k.dim() != 4, "prefix_k must be [P, Hkv, D] and k [B, S, Hkv, D] or pages")
    P, Hkv = prefix_k.shape[:2]
    device = q.device
    sq = _rows("q", q, q, (B, T, Hq, D))
    sp = _rows("prefix_k", prefix_k, q, (P, Hkv, D))
    _refuse(_rows("prefix_v", prefix_v, q, (P, Hkv, D)) != sp, "prefix_k and prefix_v must have the same strides")
    if block_table is None:
        S, page, pages, table, st = k.shape[1], 0, 0, 0, 0
        sk = _rows("k", k, q, (B, S, Hkv, D))
    else:
        pages, page = k.shape[:2]
        sk = _rows("k", k, q, (pages, page, Hkv, D))
        _refuse(block_table.dim() != 2 or block_table.shape[0] != B, "block_table must be [B, pages]")
        table = _on("block_table", block_table, torch.int32, device)
        st = block_table.shape[1]
        S = st * page
    _refuse(_rows("v", v, q, tuple(k.shape)) != sk, "k and v must have the same strides")
    n = _on("lengths", lengths, torch.int32, device, (B,))
    with _Work(device, stream) as handle:
        if out is None:
            out = torch.empty((B, T, Hq, D), dtype=q.dtype, device=device)
        o = _on("out", out, q.dtype, device, (B, T, Hq, D))
        lse = torch.empty((B, T, Hq), dtype=torch.float32, device=device) if return_lse else None
        args = _PREFIX_ARGS.pack(
            q.data_ptr(), prefix_k.data_ptr(), prefix_v.data_ptr(), k.data_ptr(), v.data_ptr(), n, table, o,
            lse.data_ptr() if return_lse else 0, code, B, T, Hq, Hkv, D, P, S, page, pages, sq[0], sq[1], sq[2],
            sp[0], sp[1], sk[0], sk[1], sk[2], st, D ** -0.5 if scale is None else scale)
        L = lib()
        ws = _workspace(L.df11_prefix_attention_workspace_bytes(args), device)
        check(L.df11_prefix_attention(args, ws.data_ptr(), ws.numel(), handle), "df11_prefix_attention")
    return (out, lse) if return_lse else out


class BoundedCache:
    """A cache of `slots` slots for each sequence and key head, of which the
    ones that gather the most attention stay.

    k, v [B, Hkv, slots, D] (bfloat16 or float16, the same strides), weights
    [B, Hkv, slots] float32, positions [B, Hkv, slots] int32, lengths [B]
    int32: the slots [0, lengths[b]) are in use.  Slots whose position is
    NO_TOKEN hold none; slots at or past a sequence's next position (refused
    drafts) are not seen and are replaced first."""

    def __init__(self, k, v, weights, positions, lengths):
        self.code = _operand("k", k)
        _refuse(k.dim() != 4, "k must be [B, Hkv, slots, D]")
        shape = B, H, C, D = tuple(k.shape)
        s = _rows("k", k, k, shape)
        _refuse(_rows("v", v, k, shape) != s, "k and v must have the same strides")
        self.k, self.v, self.weights, self.positions, self.lengths = k, v, weights, positions, lengths
        self.shape, self.device = shape, k.device
        self.args = _CACHE.pack(k.data_ptr(), v.data_ptr(),
                                _on("weights", weights, torch.float32, k.device, (B, H, C)),
                                _on("positions", positions, torch.int32, k.device, (B, H, C)),
                                _on("lengths", lengths, torch.int32, k.device, (B,)),
                                self.code, B, H, C, D, s[0], s[1], s[2])

    @classmethod
    def empty(cls, batch: int, kv_heads: int, slots: int, dim: int, dtype=torch.bfloat16, device="cuda"):
        """A cache without tokens."""
        k = torch.zeros((2, batch, kv_heads, slots, dim), dtype=dtype, device=device)
        return cls(k[0], k[1], torch.zeros((batch, kv_heads, slots), device=device),
                   torch.full((batch, kv_heads, slots), NO_TOKEN, dtype=torch.int32, device=device),
                   torch.zeros(batch, dtype=torch.int32, device=device))

    def set_lengths(self, lengths) -> None:
        """The slots in use from now on (what cache_insert returned)."""
        self.lengths.copy_(lengths)


def cache_attention(q, cache: BoundedCache, pos, *, scale: Optional[float] = None, out=None, stream=None):
    """Attention of q [B, T, Hq, D] over a bounded cache.  Query token t of
    sequence b stands at position pos[b] + t (pos [B] int32) and sees the
    used slots whose positions are at most that; cache.weights grows by the
    probabilities each slot got, summed over the tokens and the heads that
    share its key head.  Returns out [B, T, Hq, D]."""
    _refuse(q.dim() != 4, "q must be [B, T, Hq, D]")
    B, T, Hq, D = q.shape
    _refuse((B, D) != (cache.shape[0], cache.shape[3]), "q has shape %s, the cache %s" % (tuple(q.shape), cache.shape))
    device = cache.device
    sq = _rows("q", q, cache.k, (B, T, Hq, D))
    p = _on("pos", pos, torch.int32, device, (B,))
    with _Work(device, stream) as handle:
        if out is None:
            out = torch.empty((B, T, Hq, D), dtype=q.dtype, device=device)
        args = _CACHE_ARGS.pack(q.data_ptr(), p, _on("out", out, q.dtype, device, (B, T, Hq, D)), T, Hq, sq[0], sq[1],
                                sq[2], D ** -0.5 if scale is None else scale)
        L = lib()
        ws = _workspace(L.df11_cache_attention_workspace_bytes(cache.args, args), device)
        check(L.df11_cache_attention(cache.args, args, ws.data_ptr(), ws.numel(), handle), "df11_cache_attention")
    return out


def cache_insert(cache: BoundedCache, k_new, v_new, pos, recent: int, *, stream=None):
    """One token into every sequence's cache, in place: k_new, v_new
    [B, Hkv, D] at position pos[b] (pos [B] int32; a negative one: no token
    for that sequence).  While a sequence uses fewer than `slots` slots the
    next one is taken, then a stale one, then the one of least weight among
    those outside the `recent` latest positions.  Returns the slots taken
    [B, Hkv] (-1: none) and the new lengths [B], both int32; cache.lengths
    is left as it is (set_lengths)."""
    B, H, C, D = cache.shape
    s = _rows("k_new", k_new, cache.k, (B, H, D))
    _refuse(_rows("v_new", v_new, cache.k, (B, H, D)) != s, "k_new and v_new must have the same strides")
    p = _on("pos", pos, torch.int32, cache.device, (B,))
    with _Work(cache.device, stream) as handle:
        slots = torch.empty((B, H), dtype=torch.int32, device=cache.device)
        lengths = torch.empty((B,), dtype=torch.int32, device=cache.device)
        check(lib().df11_cache_insert(cache.args, k_new.data_ptr(), v_new.data_ptr(), s[0], s[1], p, recent,
                                      slots.data_ptr(), lengths.data_ptr(), handle), "df11_cache_insert")
    return slots, lengths


def cache_compact(cache: BoundedCache, pos, budget: int, recent: int, *, slots: Optional[int] = None, stream=None):
    """A new cache of `slots` slots (budget when None) with the `budget`
    slots of `cache` that are worth the most: the `recent` latest positions
    before pos[b], then the greatest weights (the lowest slot of equals), in
    slot order.  Returns it and kept [B, Hkv, slots] int32, the slots that
    were kept (-1 behind them)."""
    B, H, C, D = cache.shape
    device = cache.device
    slots = budget if slots is None else slots
    _refuse(slots < 1, "the new cache needs a slot")
    p = _on("pos", pos, torch.int32, device, (B,))
    with _Work(device, stream) as handle:
        kv = torch.empty((2, B, H, slots, D), dtype=cache.k.dtype, device=device)
        numbers = torch.empty((2, B, H, slots), dtype=torch.int32, device=device)
        cut = BoundedCache(kv[0], kv[1], torch.empty((B, H, slots), dtype=torch.float32, device=device), numbers[0],
                           torch.empty((B,), dtype=torch.int32, device=device))
        check(lib().df11_cache_compact(cache.args, p, budget, recent, cut.args, numbers[1].data_ptr(),
                                       cut.lengths.data_ptr(), handle), "df11_cache_compact")
    return cut, numbers[1]


def verify_drafts(draft_tokens, target_probs, uniforms, draft_probs=None, *, counts=None, stream=None):
    """Drafted tokens taken or refused so that what is emitted is distributed
    as the target's.  draft_tokens [B, G] int32 or int64; target_probs
    [B, G + 1, V]; draft_probs [B, G, V], or None for a drafter that is
    certain of its tokens; uniforms [B, G + 1] float32 in [0, 1): one for
    each draft, the last one for the drawn token; counts [B] int32: drafts
    of each sequence where they are fewer than G.  Probabilities in float32,
    bfloat16 or float16.  Returns tokens [B, G + 1] (the drafts taken, the
    token drawn from max(p - q, 0) or behind the last draft from p, then -1)
    and the number of drafts taken [B] int32."""
    code = _operand("target_probs", target_probs, _PROBS)
    _refuse(draft_tokens.dim() != 2 or target_probs.dim() != 3, "draft_tokens must be [B, G], target_probs [B, G + 1, V]")
    B, G = draft_tokens.shape
    V = target_probs.shape[2]
    device = target_probs.device
    if draft_tokens.dtype not in (torch.int32, torch.int64):
        raise TypeError("draft_tokens must be int32 or int64, got %s" % draft_tokens.dtype)
    d = _on("draft_tokens", draft_tokens, draft_tokens.dtype, device)
    sp = _rows("target_probs", target_probs, target_probs, (B, G + 1, V))
    sq, q = (0, 0), 0
    if draft_probs is not None:
        sq, q = _rows("draft_probs", draft_probs, target_probs, (B, G, V)), draft_probs.data_ptr()
    u = _on("uniforms", uniforms, torch.float32, device, (B, G + 1))
    n = _on("counts", counts, torch.int32, device, (B,)) if counts is not None else 0
    with _Work(device, stream) as handle:
        tokens = torch.empty((B, G + 1), dtype=draft_tokens.dtype, device=device)
        accepted = torch.empty((B,), dtype=torch.int32, device=device)
        args = _VERIFY_ARGS.pack(d, n, target_probs.data_ptr(), q, u, tokens.data_ptr(), accepted.data_ptr(), code,
                                 draft_tokens.element_size(), B, G, V, sp[0], sp[1], sq[0], sq[1])
        L = lib()
        nbytes = L.df11_verify_drafts_workspace_bytes(args)
        ws = _workspace(nbytes, device) if nbytes else None
        check(L.df11_verify_drafts(args, ws.data_ptr() if nbytes else 0, nbytes, handle), "df11_verify_drafts")
    return tokens, accepted
