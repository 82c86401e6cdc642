"""More of the quantised cache's and the logits' argument checks through the C
ABI, with no GPU work: every call here is refused before anything is launched."""
import ctypes

import pytest

from huffman_decode_df11_amd import _lib
from test_host_quantized import ARG, PTR, _attend, _cache, _logits, _read, _write


@pytest.mark.parametrize("scale", [1e38, 3e38, -1e38])
def test_scales_that_would_leave_float32_are_refused(scale):
    L, c, a = _lib.lib(), _cache(), _attend(scale=scale)
    assert L.df11_quantized_attention(ctypes.byref(c), ctypes.byref(a), PTR, 1 << 40, None) == ARG
    assert b"scale" in L.df11_last_error()


Q = 1 << 40   # an address that nothing follows


def _refused(call, *args):
    return call(*(ctypes.byref(a) for a in args)) == ARG and b"share" in _lib.lib().df11_last_error()


def _attention(c, a):
    # no workspace, which is looked at behind the memory that q and out share
    return _lib.lib().df11_quantized_attention(c, a, None, 0, None)


def _rows(q, batch, tokens, heads, dim, strides):
    return {q + 2 * (b * strides[0] + t * strides[1] + h * strides[2] + d)
            for b in range(batch) for t in range(tokens) for h in range(heads) for d in range(0, dim, 8)}


@pytest.mark.parametrize("batch,tokens,heads,strides", [
    (2, 3, 4, (768, 256, 64)), (2, 3, 4, (64, 0, 0)), (2, 3, 4, (0, 0, 64)), (3, 2, 2, (512, 256, 128)), (3, 2, 2, (128, 384, 64)),
    (1, 1, 4, (8, 8, 64)), (2, 1, 2, (1024, 8, 64)), (4, 1, 2, (2048, 0, 512)), (1, 3, 2, (0, 64, 192)), (2, 2, 2, (0, 0, 0))])
def test_out_on_q(batch, tokens, heads, strides):
    """Every place of out against q's rows, one by one."""
    own = batch * tokens * heads * 64
    need = dict(batch=batch, tokens=tokens, heads=heads, q=Q, q_batch=strides[0], q_token=strides[1], q_head=strides[2], lengths=PTR,
                block_table=PTR, table_pages=2000, table_batch=2000)
    rows = _rows(Q, batch, tokens, heads, 64, strides)
    sizes, dense = (batch, tokens, heads), (tokens * heads * 64, heads * 64, 64)
    is_q = all(n == 1 or s == d for n, s, d in zip(sizes, strides, dense))
    most = sum((n - 1) * s for n, s in zip(sizes, strides)) + 64
    for at in list(range(-own - 16, most + 16, 8)):
        out = Q + 2 * at
        shares = any(x in rows for x in range(out, out + 2 * own, 16)) and not (at == 0 and is_q)
        assert _refused(_attention, _cache(), _attend(out=out, **need)) == shares, at


def _blocks(base, pages, heads, page_stride, head_stride, own):
    return {x for p in range(pages) for h in range(heads)
            for x in range(base + p * page_stride + h * head_stride, base + p * page_stride + h * head_stride + own, 16)}


# heads in pages, pages in heads, with gaps that hold the other's blocks, and single ones
@pytest.mark.parametrize("pages,heads,page_stride,head_stride", [
    (3, 2, 1024, 512), (3, 2, 2048, 1024), (3, 2, 4096, 512), (2, 3, 512, 2048), (2, 3, 1024, 4096), (1, 4, 0, 1024), (4, 1, 1024, 0),
    (1, 1, 0, 0), (3, 3, 3584, 1024)])
@pytest.mark.parametrize("what", ["codes", "scales"])
def test_keys_and_values_that_share_memory_are_not_written(pages, heads, page_stride, head_stride, what):
    """Every place of the values against the keys' blocks, one by one: 16
    positions of 32 bytes of codes, or of two pairs of scales (128 bytes)."""
    by, own = (1, 512) if what == "codes" else (4, 128)
    strides = dict(code_page=page_stride, code_head=head_stride, scale_page=page_stride // 8, scale_head=head_stride // 8)
    keys = _blocks(Q, pages, heads, page_stride // by, head_stride // by, own)
    reach = (pages * page_stride + heads * head_stride) // by + own
    for apart in range(-reach, reach + 16, 16 * (1 if reach < 4000 else 3)):
        places = dict(k_codes=Q, v_codes=Q + (1 << 30), k_scales=Q + (2 << 30), v_scales=Q + (3 << 30))
        places["k_" + what], places["v_" + what] = Q, Q + apart
        if what == "scales":
            places["k_codes"] = Q + (2 << 30)
        shares = bool(keys & _blocks(Q + apart, pages, heads, page_stride // by, head_stride // by, own))
        c = _cache(pages=pages, kv_heads=heads, **strides, **places)
        # what is right goes on to a launch that cannot be made: more tokens than one has threads for
        w = _write(k=Q, v=Q, positions=Q, lengths=Q + 64, block_table=Q, tokens=1 << 29, k_batch=0, v_batch=0)
        L = _lib.lib()
        assert L.df11_quantized_write(ctypes.byref(c), ctypes.byref(w), None) == ARG
        assert (b"keys and values" in L.df11_last_error()) == shares, apart
        assert shares or b"one launch" in L.df11_last_error()


@pytest.mark.parametrize("dtype,size", [(_lib.DF11_FP32, 4), (_lib.DF11_BF16, 2)])
@pytest.mark.parametrize("batch,tokens,logits,out", [
    (2, 3, (30, 10), (30, 10)), (2, 3, (60, 20), (60, 20)), (2, 3, (10, 40), (10, 40)), (2, 3, (70, 10), (70, 10)), (1, 4, (0, 25), (7, 25)),
    (5, 1, (25, 3), (25, 0)), (1, 1, (5, 5), (9, 9)), (2, 3, (30, 10), (66, 20)), (2, 3, (0, 10), (30, 10)), (3, 2, (0, 0), (20, 10))])
def test_out_on_logits(batch, tokens, logits, out, dtype, size):
    """Rows of 10 tokens, every place of out against those of the logits, one by one."""
    rows = lambda base, s: {base + size * (b * s[0] + t * s[1] + i) for b in range(batch) for t in range(tokens) for i in range(10)}  # noqa: E731
    same = all(n == 1 or x == y for n, x, y in zip((batch, tokens), logits, out))
    reach = 10 + sum((n - 1) * max(x, y) for n, x, y in zip((batch, tokens), logits, out)) + 3
    for apart in range(-reach, reach + 1):
        a, b = rows(Q, logits), rows(Q + size * apart, out)
        # what is right goes on to a mask that is misaligned
        x = _logits(logits=Q, out=Q + size * apart, dtype=dtype, batch=batch, tokens=tokens, vocab=10, logits_batch=logits[0],
                    logits_token=logits[1], out_batch=out[0], out_token=out[1], mask=PTR + 2)
        shares = bool(a & b) and apart != 0 if same else max(min(a), min(b)) <= min(max(a), max(b))   # of other strides: by where all lie
        L = _lib.lib()
        assert L.df11_adjust_logits(ctypes.byref(x), None) == ARG
        assert (b"share" if shares else b"misaligned") in L.df11_last_error(), apart


def test_out_between_the_rows_of_the_logits():
    """Two halves of one allocation's rows: the same strides, nothing shared, refused for its launch only."""
    L = _lib.lib()
    x = _logits(logits=Q, out=Q + 4 * (1 << 22), batch=60000, tokens=1, vocab=1 << 22, logits_batch=1 << 23, out_batch=1 << 23, logits_token=0,
                out_token=0, history_tokens=0)
    assert L.df11_adjust_logits(ctypes.byref(x), None) == ARG and b"one launch" in L.df11_last_error()
    for change in (dict(out=Q + 4 * ((1 << 22) - 1)), dict(out=Q + 4 * ((1 << 22) + 1)), dict(out=Q - 4)):
        for n, v in change.items():
            setattr(x, n, v)
        assert L.df11_adjust_logits(ctypes.byref(x), None) == ARG and b"share" in L.df11_last_error()


def test_rows_read_back_to_one_place():
    """k and v [2, 5, 2, 64]: what shares memory is refused, and what does not for its launch only."""
    L, own = _lib.lib(), 2 * 5 * 2 * 64 * 2
    for apart in (0, 16, own - 16, 16 - own):
        r = _read(k=Q, v=Q + apart)
        assert L.df11_quantized_read(ctypes.byref(_cache()), ctypes.byref(r), None) == ARG
        assert b"k and v share memory" in L.df11_last_error()
    count = 1 << 30
    own = 2 * count * 2 * 64 * 2
    for apart, what in ((own, b"one launch"), (-own, b"one launch"), (own - 16, b"share"), (16 - own, b"share")):
        r = _read(k=Q * 4, v=Q * 4 + apart, count=count, lengths=Q)
        assert L.df11_quantized_read(ctypes.byref(_cache()), ctypes.byref(r), None) == ARG
        assert what in L.df11_last_error(), apart


@pytest.mark.parametrize("which", ["positions", "counts"])
@pytest.mark.parametrize("apart,shares", [(0, True), (4, True), (-4, True), (8, False), (-8, False)])
def test_lengths_on_what_they_are_made_of(which, apart, shares):
    """Two sequences' lengths, which one workgroup each writes, against their positions or counts."""
    L = _lib.lib()
    w = _write(k=Q, v=Q, positions=Q, counts=Q + 64, lengths=Q + (0 if which == "positions" else 64) + apart, tokens=1 << 29, k_batch=0,
               v_batch=0)
    c = _cache(k_codes=Q, v_codes=Q + (1 << 30), k_scales=Q + (2 << 30), v_scales=Q + (3 << 30))
    assert L.df11_quantized_write(ctypes.byref(c), ctypes.byref(w), None) == ARG
    assert (b"shared pointer" in L.df11_last_error()) == shares and (shares or b"one launch" in L.df11_last_error())
