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


# The checks of a call's tensors: one condition that holds where all is well,
# and behind it what names the fault.
def _fault(name: str, t, dtype, device, shape) -> None:
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if t.device != device:
        raise ValueError("%s is on %s, the other operands on %s" % (name, t.device, device))
    if t.shape != shape:
        raise ValueError("%s has shape %s, not %s" % (name, tuple(t.shape), tuple(shape)))


def _flat(name: str, t, dtype, device, shape) -> int:
    """The address of a contiguous tensor of this type, device and shape."""
    if t.dtype is dtype and t.device == device and t.shape == shape and t.is_contiguous():
        return t.data_ptr()
    _fault(name, t, dtype, device, shape)
    raise ValueError("%s must be contiguous" % name)


def _rows(name: str, t, dtype, device, shape):
    """The strides of a tensor of rows, its last axis contiguous."""
    s = t.stride()
    if t.dtype is dtype and t.device == device and t.shape == shape and s[-1] == 1 and 1 not in shape:
        return s
    _fault(name, t, dtype, device, shape)
    s = tuple(0 if n == 1 else x for n, x in zip(shape, s))   # the stride of an axis of one is never used
    if s[-1] != 1 and shape[-1] > 1:
        raise ValueError("the last axis of %s must be contiguous" % name)
    return s


def _pair(a_name: str, a, b_name: str, b, dtype, device, shape):
    """The strides of keys and values, which share them."""
    s = _rows(a_name, a, dtype, device, shape)
    if b.dtype is dtype and b.device == device and b.shape == shape and b.stride() == s:
        return s
    if _rows(b_name, b, dtype, device, shape) != s:
        raise ValueError("%s and %s must have the same strides" % (a_name, b_name))
    return s


def _code(name: str, t, table) -> int:
    if not t.is_cuda:
        raise ValueError("%s must be on the GPU" % name)
    code = table.get(t.dtype)
    if code is None:
        raise TypeError("%s must be one of %s, got %s" % (name, ", ".join(str(d) for d in table), t.dtype))
    return code


def _here(device, stream) -> bool:
    """Whether a call can go ahead on the current device's current stream."""
    return stream is None and device.index == _device()


def _there(device, stream):
    """The context in which a call's device and stream are the current ones
    (its outputs and workspaces belong to that stream)."""
    return torch.cuda.device(device) if stream is None else torch.cuda.stream(stream)


# The current device and its current stream's handle without the objects and
# checks around them (0.2 of the 2 us that torch.cuda.current_stream takes, of
# some 10 for a call).
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda index: torch.cuda.current_stream(index).cuda_stream)


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
    device, dtype = q.device, q.dtype
    if not _here(device, stream):
        with _there(device, stream):
            return prefix_attention(q, prefix_k, prefix_v, k, v, lengths, block_table=block_table, scale=scale, out=out,
                                    return_lse=return_lse)
    code = _code("q", q, _DTYPES)
    if q.dim() != 4 or prefix_k.dim() != 3 or k.dim() != 4:
        raise ValueError("q must be [B, T, Hq, D], prefix_k [P, Hkv, D] and k [B, S, Hkv, D] or pages")
    shape = B, T, Hq, D = q.shape
    P, Hkv, _ = prefix_k.shape
    sq = _rows("q", q, dtype, device, shape)
    sp = _pair("prefix_k", prefix_k, "prefix_v", prefix_v, dtype, device, (P, Hkv, D))
    if block_table is None:
        S, page, pages, table, st = k.shape[1], 0, 0, 0, 0
        sk = _pair("k", k, "v", v, dtype, device, (B, S, Hkv, D))
    else:
        pages, page = k.shape[:2]
        sk = _pair("k", k, "v", v, dtype, device, (pages, page, Hkv, D))
        if block_table.dim() != 2:
            raise ValueError("block_table must be [B, pages]")
        st = block_table.shape[1]
        table = _flat("block_table", block_table, torch.int32, device, (B, st))
        S = st * page
    n = _flat("lengths", lengths, torch.int32, device, (B,))
    if out is None:
        out = q.new_empty(shape)
        o = out.data_ptr()
    else:
        o = _flat("out", out, dtype, device, shape)
    lse = torch.empty((B, T, Hq), dtype=torch.float32, device=device) if return_lse else None
    args = _PREFIX_ARGS.pack(
        q.data_ptr(), prefix_k.data_ptr(), prefix_v.data_ptr(), k.data_ptr(), v.data_ptr(), n, table, o,
        lse.data_ptr() if return_lse else 0, code, B, T, Hq, Hkv, D, P, S, page, pages, sq[0], sq[1], sq[2],
        sp[0], sp[1], sk[0], sk[1], sk[2], st, D ** -0.5 if scale is None else scale)
    L = lib()
    nbytes = L.df11_prefix_attention_workspace_bytes(args)
    ws = lengths.new_empty((nbytes + 3) // 4)
    rc = L.df11_prefix_attention(args, ws.data_ptr(), nbytes, _stream(device.index))
    if rc:
        check(rc, "df11_prefix_attention")
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
        self.code = _code("k", k, _DTYPES)
        if k.dim() != 4:
            raise ValueError("k must be [B, Hkv, slots, D]")
        shape = B, H, C, D = k.shape
        dtype, device = k.dtype, k.device
        s = _pair("k", k, "v", v, dtype, device, shape)
        self.k, self.v, self.weights, self.positions, self.lengths = k, v, weights, positions, lengths
        self.shape, self.dtype, self.device = shape, dtype, device
        self.args = _CACHE.pack(k.data_ptr(), v.data_ptr(),
                                _flat("weights", weights, torch.float32, device, (B, H, C)),
                                _flat("positions", positions, torch.int32, device, (B, H, C)),
                                _flat("lengths", lengths, torch.int32, device, (B,)),
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
    device, dtype = cache.device, cache.dtype
    if not _here(device, stream):
        with _there(device, stream):
            return cache_attention(q, cache, pos, scale=scale, out=out)
    if q.dim() != 4:
        raise ValueError("q must be [B, T, Hq, D]")
    shape = B, T, Hq, D = q.shape
    if B != cache.shape[0] or D != cache.shape[3]:
        raise ValueError("q has shape %s, the cache %s" % (tuple(shape), tuple(cache.shape)))
    sq = _rows("q", q, dtype, device, shape)
    p = _flat("pos", pos, torch.int32, device, (B,))
    if out is None:
        out = q.new_empty(shape)
        o = out.data_ptr()
    else:
        o = _flat("out", out, dtype, device, shape)
    args = _CACHE_ARGS.pack(q.data_ptr(), p, o, T, Hq, sq[0], sq[1], sq[2], D ** -0.5 if scale is None else scale)
    L = lib()
    nbytes = L.df11_cache_attention_workspace_bytes(cache.args, args)
    ws = pos.new_empty((nbytes + 3) // 4)
    rc = L.df11_cache_attention(cache.args, args, ws.data_ptr(), nbytes, _stream(device.index))
    if rc:
        check(rc, "df11_cache_attention")
    return out


def cache_insert(cache: BoundedCache, k_new, v_new, pos, recent: int, *, stream=None):
    """One token into every sequence's cache, in place: k_new, v_new
    [B, Hkv, D] at position pos[b] (pos [B] int32; a negative one: no token
    for that sequence).  While a sequence uses fewer than `slots` slots the
    next one is taken, then a stale one, then the one of least weight among
    those outside the `recent` latest positions.  Returns the slots taken
    [B, Hkv] (-1: none) and the new lengths [B], both int32; cache.lengths
    is left as it is (set_lengths)."""
    device, dtype = cache.device, cache.dtype
    if not _here(device, stream):
        with _there(device, stream):
            return cache_insert(cache, k_new, v_new, pos, recent)
    B, H, C, D = cache.shape
    s = _pair("k_new", k_new, "v_new", v_new, dtype, device, (B, H, D))
    p = _flat("pos", pos, torch.int32, device, (B,))
    slots = pos.new_empty((B, H))
    lengths = torch.empty_like(pos)
    rc = lib().df11_cache_insert(cache.args, k_new.data_ptr(), v_new.data_ptr(), s[0], s[1], p, recent, slots.data_ptr(),
                                 lengths.data_ptr(), _stream(device.index))
    if rc:
        check(rc, "df11_cache_insert")
    return slots, lengths


def cache_compact(cache: BoundedCache, pos, budget: int, recent: int, *, slots: Optional[int] = None, stream=None):
    """A new cache of `slots` slots (budget when None) with the `budget`
    slots of `cache` that are worth the most: the `recent` latest positions
    before pos[b], then the greatest weights (the lowest slot of equals), in
    slot order.  Returns it and kept [B, Hkv, slots] int32, the slots that
    were kept (-1 behind them)."""
    device, dtype = cache.device, cache.dtype
    if not _here(device, stream):
        with _there(device, stream):
            return cache_compact(cache, pos, budget, recent, slots=slots)
    B, H, C, D = cache.shape
    slots = budget if slots is None else slots
    if slots < 1:
        raise ValueError("the new cache needs a slot")
    p = _flat("pos", pos, torch.int32, device, (B,))
    k = cache.k.new_empty((B, H, slots, D))
    kept = pos.new_empty((B, H, slots))
    cut = BoundedCache(k, torch.empty_like(k), cache.weights.new_empty((B, H, slots)), torch.empty_like(kept),
                       torch.empty_like(pos))
    rc = lib().df11_cache_compact(cache.args, p, budget, recent, cut.args, kept.data_ptr(), cut.lengths.data_ptr(),
                                  _stream(device.index))
    if rc:
        check(rc, "df11_cache_compact")
    return cut, kept


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
    device, dtype = target_probs.device, target_probs.dtype
    if not _here(device, stream):
        with _there(device, stream):
            return verify_drafts(draft_tokens, target_probs, uniforms, draft_probs, counts=counts)
    code = _code("target_probs", target_probs, _PROBS)
    if draft_tokens.dim() != 2 or target_probs.dim() != 3:
        raise ValueError("draft_tokens must be [B, G], target_probs [B, G + 1, V]")
    B, G = draft_tokens.shape
    V = target_probs.shape[2]
    kind = draft_tokens.dtype
    if kind != torch.int32 and kind != torch.int64:
        raise TypeError("draft_tokens must be int32 or int64, got %s" % kind)
    d = _flat("draft_tokens", draft_tokens, kind, device, (B, G))
    sp = _rows("target_probs", target_probs, dtype, device, (B, G + 1, V))
    if draft_probs is None:
        sq, q = (0, 0), 0
    else:
        sq, q = _rows("draft_probs", draft_probs, dtype, device, (B, G, V)), draft_probs.data_ptr()
    u = _flat("uniforms", uniforms, torch.float32, device, (B, G + 1))
    n = 0 if counts is None else _flat("counts", counts, torch.int32, device, (B,))
    tokens = draft_tokens.new_empty((B, G + 1))
    accepted = torch.empty((B,), dtype=torch.int32, device=device)
    args = _VERIFY_ARGS.pack(d, n, target_probs.data_ptr(), q, u, tokens.data_ptr(), accepted.data_ptr(), code,
                             kind.itemsize, B, G, V, sp[0], sp[1], sq[0], sq[1])
    L = lib()
    nbytes = L.df11_verify_drafts_workspace_bytes(args)
    ws = accepted.new_empty(nbytes // 4) if nbytes else None
    rc = L.df11_verify_drafts(args, ws.data_ptr() if nbytes else 0, nbytes, _stream(device.index))
    if rc:
        check(rc, "df11_verify_drafts")
    return tokens, accepted
