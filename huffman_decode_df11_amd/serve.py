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
* ``QuantizedCache``, keys and values in pages of 4-bit codes, with
  ``quantized_write`` (rows into it), ``quantized_read`` (and back) and
  ``quantized_attention`` (over it as it is);
* ``adjust_logits``     penalties for repeated tokens, biases and grammar masks;
* ``verify_drafts``     drafted tokens against the target's probabilities.

The checks of a call's tensors, its outputs, its workspace and the call into
the library are native (csrc/serve_bind.cpp); there is no fallback
implementation.  Work is enqueued on ``stream`` (the device's current stream
when None); outputs and workspaces are allocated on it.  A tensor of the
wrong type raises TypeError, one of the wrong shape, device or strides
ValueError, what the library refuses DF11Error.  There are no gradients: a
tensor that requires one raises ValueError unless gradients are off
(torch.no_grad, torch.inference_mode).
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
from typing import Optional

import torch

from . import _lib

NO_TOKEN = _lib.DF11_NO_TOKEN   # position of a cache slot that holds no token


def _load():
    path = os.path.join(os.path.dirname(os.path.abspath(__file__)), "_build", "_df11_serve.so")
    if not os.path.exists(path):
        raise ImportError("%s not found; build it with `python -m huffman_decode_df11_amd.build`" % path)
    loader = importlib.machinery.ExtensionFileLoader("_df11_serve", path)
    module = importlib.util.module_from_spec(importlib.util.spec_from_file_location("_df11_serve", path, loader=loader))
    L = _lib.lib()
    module.bind(_lib.check, *(ctypes.cast(getattr(L, "df11_" + name), ctypes.c_void_p).value for name in (
        "prefix_attention_workspace_bytes", "prefix_attention", "cache_attention_workspace_bytes", "cache_attention",
        "cache_insert", "cache_compact", "verify_drafts_workspace_bytes", "verify_drafts", "quantized_write",
        "quantized_read", "quantized_attention_workspace_bytes", "quantized_attention", "adjust_logits")))
    return module


_native = _load()

# The current device and its current stream's handle without the objects and
# checks around them (0.2 of the 2 us that torch.cuda.current_stream takes, of
# some 10 for a call).
_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda index: torch.cuda.current_stream(index).cuda_stream)


def _elsewhere(t, stream) -> bool:
    """Whether a call is meant for another device or stream than the current ones."""
    return stream is not None or (t.is_cuda and t.get_device() != _device())


def _there(t, stream):
    """The context in which a call's device and stream are the current ones
    (its outputs and workspaces belong to that stream)."""
    if stream is not None and stream.device != t.device:
        raise ValueError("the stream is of %s, the operands are on %s" % (stream.device, t.device))
    return torch.cuda.device(t.device) if stream is None else torch.cuda.stream(stream)


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
    if _elsewhere(q, stream):
        with _there(q, stream):
            return prefix_attention(q, prefix_k, prefix_v, k, v, lengths, block_table=block_table, scale=scale, out=out,
                                    return_lse=return_lse)
    return _native.prefix_attention(q, prefix_k, prefix_v, k, v, lengths, block_table, scale, out, return_lse,
                                    _stream(_device()))


class BoundedCache:
    """A cache of `slots` slots for each sequence and key head, of which the
    ones that gather the most attention stay.

    k, v [B, Hkv, slots, D] (bfloat16 or float16, the same strides), weights
    [B, Hkv, slots] float32, positions [B, Hkv, slots] int32, lengths [B]
    int32: the slots [0, lengths[b]) are in use.  Slots whose position is
    NO_TOKEN hold none; slots at or past a sequence's next position (refused
    drafts) are not seen and are replaced first."""

    def __init__(self, k, v, weights, positions, lengths):
        # args: the tensors as the binding takes them, which reads their addresses and checks them in every call
        self.__dict__.update(k=k, v=v, weights=weights, positions=positions, lengths=lengths,
                             args=_native.cache(k, v, weights, positions, lengths))

    def __setattr__(self, name, value):
        raise AttributeError("a BoundedCache keeps its tensors: write into %s, or make another cache" % name)

    @property
    def shape(self):
        """(B, Hkv, slots, D)"""
        return self.k.shape

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

    def forget(self, pos, *, stream=None) -> None:
        """Tokens taken back, in place: every slot whose position is pos[b] or
        more holds no token from now on (pos [B] int32, the sequence's next
        position; a negative one: that sequence keeps all).  To be called
        whenever drafts that were inserted are refused: left as they are,
        they would be seen again, beside the tokens that took their
        positions, as soon as the sequence has passed them.  The weights that
        the refused tokens' queries gave other slots stay."""
        if _elsewhere(self.k, stream):
            with _there(self.k, stream):
                return self.forget(pos)
        if not isinstance(pos, torch.Tensor) or pos.dtype != torch.int32:
            raise TypeError("pos must be an int32 tensor")
        if pos.device != self.positions.device or tuple(pos.shape) != (self.shape[0],):
            raise ValueError("pos must be [%d] on %s" % (self.shape[0], self.positions.device))
        at = pos.view(-1, 1, 1)
        self.positions.masked_fill_((self.positions >= at) & (at >= 0), NO_TOKEN)


def cache_attention(q, cache: BoundedCache, pos, *, scale: Optional[float] = None, out=None, stream=None):
    """Attention of q [B, T, Hq, D] over a bounded cache.  Query token t of
    sequence b stands at position pos[b] + t (pos [B] int32) and sees the
    used slots whose positions are at most that; cache.weights grows by the
    probabilities each slot got, summed over the tokens and the heads that
    share its key head.  Returns out [B, T, Hq, D]."""
    if _elsewhere(cache.k, stream):
        with _there(cache.k, stream):
            return cache_attention(q, cache, pos, scale=scale, out=out)
    return _native.cache_attention(cache.args, cache.k, q, pos, scale, out, _stream(_device()))


def cache_insert(cache: BoundedCache, k_new, v_new, pos, recent: int, *, stream=None):
    """One token into every sequence's cache, in place: k_new, v_new
    [B, Hkv, D] at position pos[b] (pos [B] int32; a negative one: no token
    for that sequence).  While a sequence uses fewer than `slots` slots the
    next one is taken, then the first stale one (without a token, or at pos[b]
    or past it), then the one of least weight among those outside the `recent`
    latest positions.  No other slot changes: BoundedCache.forget gives up
    tokens that were taken back.  Returns the slots taken
    [B, Hkv] (-1: none) and the new lengths [B], both int32; cache.lengths
    is left as it is (set_lengths)."""
    if _elsewhere(cache.k, stream):
        with _there(cache.k, stream):
            return cache_insert(cache, k_new, v_new, pos, recent)
    return _native.cache_insert(cache.args, cache.k, k_new, v_new, pos, recent, _stream(_device()))


def cache_compact(cache: BoundedCache, pos, budget: int, recent: int, *, slots: Optional[int] = None, stream=None):
    """A new cache of `slots` slots (budget when None) with the `budget`
    slots of `cache` that are worth the most: the `recent` latest positions
    before pos[b], then the greatest weights (the lowest slot of equals), in
    slot order.  Returns it and kept [B, Hkv, slots] int32, the slots that
    were kept (-1 behind them)."""
    if _elsewhere(cache.k, stream):
        with _there(cache.k, stream):
            return cache_compact(cache, pos, budget, recent, slots=slots)
    *parts, kept = _native.cache_compact(cache.args, cache.k, pos, budget, recent, budget if slots is None else slots,
                                         _stream(_device()))
    return BoundedCache(*parts), kept


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
    if _elsewhere(target_probs, stream):
        with _there(target_probs, stream):
            return verify_drafts(draft_tokens, target_probs, uniforms, draft_probs, counts=counts)
    return _native.verify_drafts(draft_tokens, target_probs, uniforms, draft_probs, counts, _stream(_device()))


class QuantizedCache:
    """A cache of pages whose keys and values are held in 4 bits.

    k_codes, v_codes [pages, Hkv, page, D / 2] uint8: dim 2 i in the low half
    of byte i.  k_scales, v_scales [pages, Hkv, page, G, 2] (bfloat16 or
    float16, the type of the rows that are written and read): the step and the
    least value of each of a row's G groups, G = 2 for D up to 64 and 4 above,
    dim d in group d % G; a code stands for code * step + least.  page is a
    multiple of 16, D a multiple of 8 up to 256.  Pages and heads may have any
    strides, a head's positions in a page lie one behind the other."""

    def __init__(self, k_codes, v_codes, k_scales, v_scales):
        # args: the tensors as the binding takes them, which reads their addresses and checks them in every call
        self.__dict__.update(k_codes=k_codes, v_codes=v_codes, k_scales=k_scales, v_scales=v_scales,
                             args=_native.quantized(k_codes, v_codes, k_scales, v_scales))

    def __setattr__(self, name, value):
        raise AttributeError("a QuantizedCache keeps its tensors: write into %s, or make another cache" % name)

    @property
    def shape(self):
        """(pages, Hkv, page, D)"""
        pages, heads, page, half = self.k_codes.shape
        return torch.Size((pages, heads, page, 2 * half))

    @classmethod
    def empty(cls, pages: int, kv_heads: int, page: int, dim: int, dtype=torch.bfloat16, device="cuda"):
        """A cache whose rows are all zero."""
        codes = torch.zeros((2, pages, kv_heads, page, dim // 2), dtype=torch.uint8, device=device)
        scales = torch.zeros((2, pages, kv_heads, page, 2 if dim <= 64 else 4, 2), dtype=dtype, device=device)
        return cls(codes[0], codes[1], scales[0], scales[1])


def quantized_write(cache: QuantizedCache, k, v, positions, *, counts=None, block_table=None, stream=None):
    """New rows into a quantised cache, in place: token t of sequence b, k and
    v [B, T, Hkv, D] in the cache's type, goes to position positions[b] + t
    (positions [B] int32).  counts [B] int32: the first counts[b] tokens of a
    sequence, all T when None.  Position s of sequence b is row s % page of
    page block_table[b, s // page] (int32; page b alone when None); what lies
    outside the table or the cache is not written.  A group of values with a
    NaN or an infinity among them becomes NaN.  No two tokens of a call may go
    to the same row, and the cache's keys and values share no memory.  Returns the lengths behind the new tokens, positions +
    counts [B] int32."""
    if _elsewhere(cache.k_codes, stream):
        with _there(cache.k_codes, stream):
            return quantized_write(cache, k, v, positions, counts=counts, block_table=block_table)
    return _native.quantized_write(cache.args, k, v, positions, counts, block_table, _stream(_device()))


def quantized_read(cache: QuantizedCache, lengths, count: int, *, first=None, block_table=None, out=None, stream=None):
    """`count` positions of every sequence back as 16-bit rows, from first[b]
    on (int32; 0 when None): k, v [B, count, Hkv, D], zeros from lengths[b]
    (int32) on and where the table holds no page.  A code that stands for more
    than the type's greatest number is read as that.  out: a pair of such
    tensors to write to, which share no memory."""
    if _elsewhere(cache.k_codes, stream):
        with _there(cache.k_codes, stream):
            return quantized_read(cache, lengths, count, first=first, block_table=block_table, out=out)
    return _native.quantized_read(cache.args, lengths, count, first, block_table, out, _stream(_device()))


def quantized_attention(q, cache: QuantizedCache, lengths, *, block_table=None, scale: Optional[float] = None, out=None,
                        return_lse: bool = False, stream=None):
    """Attention over a quantised cache, whose values are taken as their codes
    stand for them.  q [B, T, Hq, D]: the last T of each sequence's lengths[b]
    positions (int32); token t sees the first lengths - T + 1 + t of them.
    Returns out [B, T, Hq, D] (which may be q itself, but shares no other memory
    with it), and with return_lse also lse [B, T, Hq]
    float32.  A row that sees no position is zero (lse -inf).  Values of V stay
    below 2^115 / lengths in size: past that up to 112 rows may come out infinite or NaN."""
    if _elsewhere(cache.k_codes, stream):
        with _there(cache.k_codes, stream):
            return quantized_attention(q, cache, lengths, block_table=block_table, scale=scale, out=out, return_lse=return_lse)
    return _native.quantized_attention(cache.args, q, lengths, block_table, scale, out, return_lse, _stream(_device()))


def adjust_logits(logits, history=None, lengths=None, *, prompt_lengths=None, drafts=None, repetition=None, presence=None,
                  frequency=None, bias=None, mask=None, out=None, stream=None):
    """A request's wishes on the logits of its next tokens: logits [B, T, V]
    or [B, V], float32, bfloat16 or float16.

    history [B, L] with lengths [B]: the tokens that a sequence holds, the
    first prompt_lengths[b] of them (none when None) its prompt; drafts
    [B, T - 1]: what stands before the rows behind the first, row t having
    seen drafts[:, :t].  A token seen anywhere has its logit divided by
    repetition[b] if positive, multiplied if not; one that was said n > 0
    times outside the prompt loses frequency[b] * n + presence[b]; bias =
    (tokens [B, N], values [B, N] float32) adds to the tokens listed (those
    outside the vocabulary, -1 for one, to none).  mask [B, T, ceil(V / 32)]
    int32 ([B, ceil(V / 32)] for logits [B, V]): a token whose bit is 0 gets
    -inf; a row may have none left.  Tokens int32 or int64, all alike;
    lengths int32; repetition, presence and frequency [B] float32.  Returns
    out, which may be logits itself, but shares no other memory with it."""
    if _elsewhere(logits, stream):
        with _there(logits, stream):
            return adjust_logits(logits, history, lengths, prompt_lengths=prompt_lengths, drafts=drafts, repetition=repetition,
                                 presence=presence, frequency=frequency, bias=bias, mask=mask, out=out)
    tokens, values = (None, None) if bias is None else bias
    return _native.adjust_logits(logits, history, lengths, prompt_lengths, drafts, repetition, presence, frequency, tokens,
                                 values, mask, out, _stream(_device()))
