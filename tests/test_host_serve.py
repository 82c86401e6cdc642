"""The generation operators' argument checks through the C ABI and the
binding, with no GPU work: every call here is refused before anything is
launched, so its pointers (host memory) are never followed on the device."""
import ctypes

import numpy as np
import pytest

from huffman_decode_df11_amd import _lib

ARG = -1
_HELD = np.zeros(4096 + 64, np.uint8)
PTR = _HELD.ctypes.data + (-_HELD.ctypes.data) % 64


def _prefix(**change):
    a = _lib.PrefixAttentionArgs(q=PTR, prefix_k=PTR, prefix_v=PTR, k=PTR, v=PTR, lengths=PTR, out=PTR, dtype=_lib.DF11_BF16,
                                 batch=2, tokens=1, heads=8, kv_heads=2, dim=64, prefix=100, suffix=32, q_batch=512,
                                 q_token=512, q_head=64, prefix_token=128, prefix_head=64, k_batch=4096, k_token=128,
                                 k_head=64, scale=0.125)
    for n, v in change.items():
        setattr(a, n, v)
    return a


def _cache(**change):
    c = _lib.Cache(k=PTR, v=PTR, weights=PTR, positions=PTR, lengths=PTR, dtype=_lib.DF11_FP16, batch=2, kv_heads=2, slots=40,
                   dim=64, stride_batch=5120, stride_head=2560, stride_slot=64)
    for n, v in change.items():
        setattr(c, n, v)
    return c


def _attend(**change):
    a = _lib.CacheAttentionArgs(q=PTR, pos=PTR, out=PTR, tokens=1, heads=8, q_batch=512, q_token=512, q_head=64, scale=0.125)
    for n, v in change.items():
        setattr(a, n, v)
    return a


def _verify(**change):
    a = _lib.VerifyArgs(draft_tokens=PTR, target_probs=PTR, draft_probs=PTR, uniforms=PTR, tokens=PTR, accepted=PTR,
                        dtype=_lib.DF11_FP32, token_bytes=4, batch=2, drafts=3, vocab=50000, target_batch=200000,
                        target_row=50000, draft_batch=150000, draft_row=50000)
    for n, v in change.items():
        setattr(a, n, v)
    return a


def test_structs_are_made_of_eight_byte_fields():
    for s, n in ((_lib.PrefixAttentionArgs, 29), (_lib.Cache, 13), (_lib.CacheAttentionArgs, 9), (_lib.VerifyArgs, 16)):
        assert ctypes.sizeof(s) == 8 * n == 8 * len(s._fields_)


@pytest.mark.parametrize("change", [
    dict(dtype=_lib.DF11_FP32), dict(dtype=7), dict(dim=60), dict(dim=0), dict(dim=264), dict(heads=7), dict(kv_heads=0),
    dict(heads=0, kv_heads=1), dict(batch=-1), dict(tokens=0), dict(batch=1 << 29, tokens=64), dict(prefix=-1),
    dict(prefix=1 << 31), dict(suffix=-1), dict(block_table=PTR, page=0, n_pages=4), dict(block_table=PTR, page=5, n_pages=4),
    dict(q_head=60), dict(k_token=-64), dict(prefix_token=1 << 27), dict(table_batch=-1), dict(scale=0.0), dict(scale=-1.0),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(scale=1e-60)])
def test_prefix_attention_refuses(change):
    L, a = _lib.lib(), _prefix(**change)
    assert L.df11_prefix_attention_workspace_bytes(ctypes.byref(a)) == 0
    assert L.df11_prefix_attention(ctypes.byref(a), PTR, 1 << 40, None) == ARG, L.df11_last_error()


@pytest.mark.parametrize("change", [dict(q=None), dict(out=PTR + 8), dict(k=PTR + 2), dict(prefix_v=None), dict(lengths=None)])
def test_prefix_attention_refuses_pointers(change):
    L, a = _lib.lib(), _prefix(**change)
    need = L.df11_prefix_attention_workspace_bytes(ctypes.byref(a))
    assert need > 0
    assert L.df11_prefix_attention(ctypes.byref(a), PTR, need, None) == ARG


def test_workspaces_are_checked():
    L = _lib.lib()
    a, c, t, v = _prefix(), _cache(), _attend(), _verify()
    need = L.df11_prefix_attention_workspace_bytes(ctypes.byref(a))
    assert L.df11_prefix_attention(ctypes.byref(a), PTR, need - 1, None) == ARG
    assert L.df11_prefix_attention(ctypes.byref(a), PTR + 4, need, None) == ARG
    assert L.df11_prefix_attention(ctypes.byref(a), None, need, None) == ARG
    need = L.df11_cache_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(t))
    assert need > 0 and L.df11_cache_attention(ctypes.byref(c), ctypes.byref(t), PTR, need - 1, None) == ARG
    need = L.df11_verify_drafts_workspace_bytes(ctypes.byref(v))
    assert need > 0 and L.df11_verify_drafts(ctypes.byref(v), PTR, need - 1, None) == ARG
    assert b"workspace" in L.df11_last_error()


def test_null_arguments_and_empty_batches():
    L = _lib.lib()
    assert L.df11_prefix_attention(None, PTR, 1 << 20, None) == ARG
    assert L.df11_cache_attention(None, None, PTR, 1 << 20, None) == ARG
    assert L.df11_cache_insert(None, PTR, PTR, 64, 64, PTR, 1, PTR, PTR, None) == ARG
    assert L.df11_cache_compact(None, PTR, 4, 1, None, PTR, PTR, None) == ARG
    assert L.df11_verify_drafts(None, PTR, 1 << 20, None) == ARG
    # nothing to do: nothing is launched, no pointer is needed
    assert L.df11_prefix_attention(ctypes.byref(_prefix(batch=0, q=None, out=None)), None, 0, None) == 0
    empty = _cache(batch=0)
    assert L.df11_cache_attention(ctypes.byref(empty), ctypes.byref(_attend()), None, 0, None) == 0
    assert L.df11_cache_insert(ctypes.byref(empty), None, None, 0, 0, None, 1, None, None, None) == 0
    assert L.df11_cache_compact(ctypes.byref(empty), None, 4, 1, ctypes.byref(empty), None, None, None) == 0
    assert L.df11_verify_drafts(ctypes.byref(_verify(batch=0)), None, 0, None) == 0


BAD_CACHES = [dict(dtype=_lib.DF11_FP32), dict(dim=12), dict(dim=512), dict(kv_heads=0), dict(batch=70000), dict(slots=-1),
              dict(stride_slot=60), dict(stride_head=-8), dict(slots=1 << 31)]


@pytest.mark.parametrize("change", BAD_CACHES)
def test_caches_are_checked(change):
    L, c = _lib.lib(), _cache(**change)
    assert L.df11_cache_attention_workspace_bytes(ctypes.byref(c), ctypes.byref(_attend())) == 0
    assert L.df11_cache_attention(ctypes.byref(c), ctypes.byref(_attend()), PTR, 1 << 40, None) == ARG
    assert L.df11_cache_insert(ctypes.byref(c), PTR, PTR, 128, 64, PTR, 1, PTR, PTR + 64, None) == ARG
    assert L.df11_cache_compact(ctypes.byref(c), PTR, 4, 1, ctypes.byref(_cache()), PTR, PTR + 64, None) == ARG
    assert L.df11_cache_compact(ctypes.byref(_cache()), PTR, 4, 1, ctypes.byref(c), PTR, PTR + 64, None) == ARG


@pytest.mark.parametrize("change", [dict(heads=7), dict(tokens=0), dict(tokens=70000), dict(q_batch=-8), dict(scale=-0.5)])
def test_cache_attention_refuses(change):
    L = _lib.lib()
    assert L.df11_cache_attention(ctypes.byref(_cache()), ctypes.byref(_attend(**change)), PTR, 1 << 40, None) == ARG


def test_cache_insert_refuses():
    L, c = _lib.lib(), _cache()
    assert L.df11_cache_insert(ctypes.byref(c), PTR, PTR, 128, 64, PTR, -1, PTR, PTR + 64, None) == ARG
    assert L.df11_cache_insert(ctypes.byref(c), PTR + 2, PTR, 128, 64, PTR, 1, PTR, PTR + 64, None) == ARG
    assert L.df11_cache_insert(ctypes.byref(c), PTR, PTR, 12, 64, PTR, 1, PTR, PTR + 64, None) == ARG
    assert L.df11_cache_insert(ctypes.byref(c), PTR, PTR, 128, 64, PTR, 1, PTR, PTR, None) == ARG   # lengths in place
    assert L.df11_cache_insert(ctypes.byref(c), PTR, PTR, 128, 64, None, 1, PTR, PTR + 64, None) == ARG


def test_cache_compact_refuses():
    L, c, out = _lib.lib(), _cache(), _cache(slots=10, k=PTR + 64, v=PTR + 64, weights=PTR + 64, positions=PTR + 64)
    call = lambda budget, recent, o: L.df11_cache_compact(ctypes.byref(c), PTR, budget, recent, ctypes.byref(o), PTR,   # noqa: E731
                                                          PTR + 64, None)
    assert call(0, 0, out) == ARG
    assert call(4, 5, out) == ARG
    assert call(4, -1, out) == ARG
    assert call(11, 1, out) == ARG
    assert call(4, 1, _cache(slots=10)) == ARG                       # in place
    for change in (dict(batch=3), dict(kv_heads=1), dict(dim=128), dict(dtype=_lib.DF11_BF16)):
        assert call(4, 1, _cache(slots=10, k=PTR + 64, v=PTR + 64, weights=PTR + 64, positions=PTR + 64, **change)) == ARG


@pytest.mark.parametrize("change", [
    dict(dtype=3), dict(token_bytes=2), dict(batch=-1), dict(batch=70000), dict(drafts=-1), dict(drafts=1025), dict(vocab=0),
    dict(vocab=(1 << 22) + 1), dict(target_row=-1), dict(target_probs=None), dict(target_probs=PTR + 2), dict(draft_probs=PTR + 1),
    dict(uniforms=None), dict(tokens=None), dict(accepted=None), dict(draft_tokens=None)])
def test_verify_drafts_refuses(change):
    L = _lib.lib()
    assert L.df11_verify_drafts(ctypes.byref(_verify(**change)), PTR, 1 << 40, None) == ARG


def test_binding_refuses_what_is_not_on_the_gpu():
    torch = pytest.importorskip("torch")
    from huffman_decode_df11_amd import serve
    z = torch.zeros
    q, p, k = z(2, 1, 4, 64, dtype=torch.bfloat16), z(9, 2, 64, dtype=torch.bfloat16), z(2, 8, 2, 64, dtype=torch.bfloat16)
    n = z(2, dtype=torch.int32)
    native = serve._native
    with pytest.raises(ValueError, match="on the GPU"):
        native.prefix_attention(q, p, p, k, k, n, None, None, None, False, 0)
    with pytest.raises(ValueError, match="on the GPU"):
        native.cache(k, k, z(2, 8, 2), z(2, 8, 2, dtype=torch.int32), n)
    with pytest.raises(ValueError, match="on the GPU"):
        native.verify_drafts(z(2, 3, dtype=torch.int32), z(2, 4, 50), z(2, 4), None, None, 0)
    with pytest.raises(TypeError, match="must be a tensor"):
        native.prefix_attention(q, None, p, k, k, n, None, None, None, False, 0)
    with pytest.raises(TypeError, match="not a BoundedCache"):
        native.cache_attention(b"", k, q, n, None, None, 0)
    with pytest.raises(TypeError, match="arguments"):
        native.verify_drafts(n)


@pytest.mark.parametrize("change", [dict(stride_head=0), dict(stride_batch=0), dict(stride_slot=0), dict(stride_slot=56),
                                    dict(stride_head=2552), dict(stride_batch=2560), dict(stride_batch=64)])
def test_caches_whose_slots_share_memory_are_not_written(change):
    L = _lib.lib()
    assert L.df11_cache_insert(ctypes.byref(_cache(**change)), PTR, PTR, 128, 64, PTR, 1, PTR, PTR + 64, None) == ARG
    out = _cache(k=PTR + 64, v=PTR + 64, weights=PTR + 64, positions=PTR + 64, **change)
    assert L.df11_cache_compact(ctypes.byref(_cache()), PTR, 4, 1, ctypes.byref(out), PTR, PTR + 64, None) == ARG
    assert b"share memory" in L.df11_last_error()


@pytest.mark.parametrize("change", [dict(k=PTR + 64), dict(v=PTR + 64), dict(k=PTR + (1 << 20) - 64), dict(weights=PTR + 16),
                                    dict(positions=PTR + (1 << 20) + 48), dict(weights=PTR - 64)])
def test_caches_that_lie_on_each_other_are_not_cut_down(change):
    """Each part of the new cache that begins inside the old one, or ends in it."""
    far = 1 << 20   # nothing here is followed: the old cache holds 2 * 2 * 40 slots of 64 dims
    old = _cache(v=PTR + far, positions=PTR + far)
    apart = dict(slots=10, k=PTR + 2 * far, v=PTR + 3 * far, weights=PTR + 2 * far, positions=PTR + 3 * far,
                 stride_batch=1280, stride_head=640)
    L = _lib.lib()
    out = _cache(**{**apart, **change})
    assert L.df11_cache_compact(ctypes.byref(old), PTR, 4, 1, ctypes.byref(out), PTR, PTR + 64, None) == ARG
    assert b"in place" in L.df11_last_error()


def test_attention_of_more_workgroups_than_a_launch_has_is_refused():
    """Rows past what one launch joins (2^24 workgroups of four): refused before the first launch."""
    L = _lib.lib()
    a = _prefix(batch=1 << 10, tokens=1 << 12, heads=1 << 8, kv_heads=2, dim=8)
    assert L.df11_prefix_attention_workspace_bytes(ctypes.byref(a)) > 0
    assert L.df11_prefix_attention(ctypes.byref(a), PTR, (1 << 63) - 1, None) == ARG
    c = _cache(batch=1 << 10)
    t = _attend(tokens=1 << 12, heads=1 << 8)
    assert L.df11_cache_attention(ctypes.byref(c), ctypes.byref(t), PTR, (1 << 63) - 1, None) == ARG
    assert b"one launch" in L.df11_last_error()
