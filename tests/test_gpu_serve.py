"""The generation operators on the GPU against their definitions in 64 bits
(serve_reference.py): types, head layouts, lengths from none to several
workgroups' ranges, page sizes, strides, masked places that hold NaN and
infinities, rows that see nothing, streams and graphs."""
import copy
import pickle

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import serve_reference as ref  # noqa: E402
from huffman_decode_df11_amd import serve  # noqa: E402

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
INF, NAN = float("inf"), float("nan")


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _randn(g, *shape, dtype=BF):
    return torch.randn(shape, generator=g).to(dtype)


def _close(got, want, bound, what):
    got = got.cpu().double()
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), what
    off = (got - want).abs() - bound
    assert float(torch.where(torch.isfinite(want), off, -1.0).max()) <= 1e-30, (what, float(off.max()))


def _lse_close(got, want):
    got = got.cpu().double()
    assert torch.equal(got == -INF, want == -INF)
    fine = want != -INF
    assert float((got - want)[fine].abs().max() if fine.any() else 0.0) <= 2.0 ** -12


def _prefix_case(seed, B, T, P, lengths, Hq, H, D, dtype, page=0, S=None):
    g = _gen(seed)
    S = max([1] + [int(x) for x in lengths]) if S is None else S
    x = dict(q=_randn(g, B, T, Hq, D, dtype=dtype), pk=_randn(g, P, H, D, dtype=dtype), pv=_randn(g, P, H, D, dtype=dtype),
             lengths=torch.tensor(lengths, dtype=torch.int32), table=None)
    if page:
        per = -(-S // page)
        x["k"], x["v"] = _randn(g, B * per + 2, page, H, D, dtype=dtype), _randn(g, B * per + 2, page, H, D, dtype=dtype)
        x["table"] = (torch.randperm(B * per + 2, generator=g)[:B * per]).view(B, per).to(torch.int32)
    else:
        x["k"], x["v"] = _randn(g, B, S, H, D, dtype=dtype), _randn(g, B, S, H, D, dtype=dtype)
    return x


def _run_prefix(x, **more):
    c = {n: t.cuda() if t is not None else None for n, t in x.items()}
    return serve.prefix_attention(c["q"], c["pk"], c["pv"], c["k"], c["v"], c["lengths"], block_table=c["table"],
                                  return_lse=True, **more)


def _check_prefix(x, what, **more):
    print("case", what, flush=True)
    out, lse = _run_prefix(x, **more)
    torch.cuda.synchronize()
    want, want_lse, bound = ref.prefix_attention(x["q"], x["pk"], x["pv"], x["k"], x["v"], x["lengths"], x["table"],
                                                 more.get("scale"))
    assert out.dtype == x["q"].dtype and lse.dtype == F32
    _close(out, want, bound, what)
    _lse_close(lse, want_lse)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("B,T,P,lengths,Hq,H,D,page", [
    (1, 1, 0, [1], 1, 1, 8, 0),
    (1, 1, 1, [0], 2, 1, 64, 0),
    (2, 1, 31, [1, 40], 8, 2, 128, 0),
    (3, 2, 32, [2, 33, 5], 6, 2, 72, 0),
    (2, 1, 33, [7, 129], 7, 1, 96, 7),
    (5, 4, 257, [4, 16, 17, 300, 31], 8, 2, 128, 16),
    (1, 17, 100, [17], 4, 4, 64, 64),
    (2, 9, 640, [9, 50], 40, 1, 80, 16),
    (4, 1, 1100, [3, 0, 64, 65], 12, 12, 64, 0),
    (2, 3, 129, [3, 200], 6, 3, 256, 16),
    (1, 2, 70, [70], 4, 2, 200, 1),
])
def test_prefix_attention(B, T, P, lengths, Hq, H, D, page, dtype):
    _check_prefix(_prefix_case(B * 100 + T + D, B, T, P, lengths, Hq, H, D, dtype, page), (B, T, P, lengths, Hq, H, D, page))


def test_prefix_attention_many_rows_long_prefix():
    """More rows than a tile and a prefix of several ranges."""
    _check_prefix(_prefix_case(5, 37, 1, 2500, [1 + (7 * i) % 90 for i in range(37)], 8, 2, 128, BF, 16), "37 x 2500")


@pytest.mark.parametrize("B,T,P,S,Hq,H,D", [(33, 4, 40, 20, 8, 2, 64), (5, 1, 32768, 9, 64, 16, 8), (2, 1, 5000, 1100, 2, 1, 128)])
def test_prefix_attention_row_counts_and_ranges(B, T, P, S, Hq, H, D):
    """Enough rows for four to a joining workgroup; a prefix that is nearly
    all there is; few rows of many ranges."""
    _check_prefix(_prefix_case(B + P, B, T, P, [T + (i * 7) % (S - T + 1) for i in range(B)], Hq, H, D, BF, S=S),
                  (B, T, P, S, Hq, H, D))


def test_offsets_past_32_bits():
    """Pages, sequences and slots whose elements lie more than 2^32 bytes and
    2^31 elements into their tensors."""
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of device memory")
    pages = 140_000   # of 16 positions, 8 heads, 128 dims: 2.3e9 elements
    x = _prefix_case(14, 2, 1, 30, [40, 33], 16, 8, 128, BF, 16, S=48)
    k, v = (torch.empty((pages, 16, 8, 128), dtype=BF, device="cuda") for _ in range(2))
    table = x["table"].clone()
    for i, p in enumerate(x["table"].flatten().tolist()):
        at = pages - 1 - i
        k[at], v[at] = x["k"][p].cuda(), x["v"][p].cuda()
        table.view(-1)[i] = at
    out, lse = serve.prefix_attention(x["q"].cuda(), x["pk"].cuda(), x["pv"].cuda(), k, v, x["lengths"].cuda(),
                                      block_table=table.cuda(), return_lse=True)
    want, want_lse, bound = ref.prefix_attention(x["q"], x["pk"], x["pv"], x["k"], x["v"], x["lengths"], x["table"])
    _close(out, want, bound, "pages")
    _lse_close(lse, want_lse)
    # the same memory as caches of two sequences, the second 2^31 elements behind the first
    y = _cache_case(15, 2, 2, 70, 128, [70, 70], more=5)
    far = 1 << 31
    flat_k, flat_v = k.view(-1), v.view(-1)
    strides = (far, 70 * 128, 128, 1)
    ck, cv = (t.as_strided((2, 2, 70, 128), strides) for t in (flat_k, flat_v))
    ck.copy_(y["k"])
    cv.copy_(y["v"])
    cache = serve.BoundedCache(ck, cv, y["weights"].cuda(), y["positions"].cuda(), y["lengths"].cuda())
    q, pos = _randn(_gen(8), 2, 1, 4, 128), torch.tensor([75, 74], dtype=torch.int32)
    cut, kept = serve.cache_compact(cache, pos.cuda(), 20, 4)
    assert torch.equal(kept.cpu(), ref.cache_compact(y["positions"], y["weights"], y["lengths"], pos, 20, 4))
    rows = kept.cpu().long().unsqueeze(-1).expand(2, 2, 20, 128)
    assert torch.equal(cut.k.cpu(), y["k"].gather(2, rows)) and torch.equal(cut.v.cpu(), y["v"].gather(2, rows))
    want, want_w, bound = ref.cache_attention(q, pos=pos, **y)
    _close(serve.cache_attention(q.cuda(), cache, pos.cuda()), want, bound, "cache")
    _close(cache.weights, want_w, 2.0 ** -12 * (want_w - y["weights"].double()) + 2.0 ** -22 * want_w, "weights")
    window = _randn(_gen(9), 2, 20, 4, 128)
    want, _, bound = ref.cache_attention(window, pos=pos - 19, **y)
    _close(serve.cache_attention(window.cuda(), cache, pos.cuda() - 19), want, bound, "window")
    slots, _ = ref.cache_insert(y["positions"], cache.weights.cpu(), y["lengths"], pos, 4)
    row = _randn(_gen(10), 2, 2, 128)
    got, _ = serve.cache_insert(cache, row.cuda(), row.cuda(), pos.cuda(), 4)
    assert torch.equal(got.cpu(), slots)
    for b in range(2):
        for h in range(2):
            assert torch.equal(ck[b, h, int(slots[b, h])].cpu(), row[b, h])


def test_prefix_attention_empty_rows_and_scale():
    """No prefix: query tokens before the first own position see nothing."""
    x = _prefix_case(6, 4, 3, 0, [0, 1, 2, 3], 4, 2, 64, BF, S=8)
    out, lse = _run_prefix(x)
    assert bool((out[0] == 0).all()) and bool((lse[0] == -INF).all())
    assert bool((out[1, :2] == 0).all()) and bool((lse[1, 2] > -INF).all())
    _check_prefix(x, "empty rows")
    _check_prefix(_prefix_case(7, 2, 1, 50, [9, 20], 4, 2, 64, HF), "scale", scale=0.3)


def test_prefix_attention_lengths_are_clamped():
    x = _prefix_case(8, 3, 1, 20, [5, 9, 16], 4, 2, 64, BF, S=16)
    x["lengths"] = torch.tensor([-3, 9, 99], dtype=torch.int32)
    _check_prefix(x, "clamped")


@pytest.mark.parametrize("page", [0, 16, 5])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_prefix_attention_masked_places_hold_anything(bad, page, dtype):
    """Positions behind a sequence's length, and unused pages, hold `bad`."""
    lengths = [3, 17, 40, 64]
    x = _prefix_case(9, 4, 3, 65, lengths, 8, 2, 128, dtype, page, S=70)
    clean = {n: t.clone() if t is not None else None for n, t in x.items()}
    if page:
        used = torch.zeros(x["k"].shape[:2], dtype=torch.bool)
        for b, n in enumerate(lengths):
            for s in range(n):
                used[int(x["table"][b, s // page]), s % page] = True
    else:
        used = torch.arange(70)[None] < torch.tensor(lengths)[:, None]
    for name in ("k", "v"):
        x[name][~used] = bad
        clean[name][~used] = 0
    out, lse = _run_prefix(x)
    want, want_lse, bound = ref.prefix_attention(clean["q"], clean["pk"], clean["pv"], clean["k"], clean["v"],
                                                 clean["lengths"], clean["table"])
    _close(out, want, bound, "masked")
    _lse_close(lse, want_lse)


@pytest.mark.parametrize("bad", [NAN, INF])
def test_prefix_attention_later_drafts_do_not_reach_earlier_ones(bad):
    """The last drafted position holds `bad`: only the last token sees it."""
    x = _prefix_case(10, 2, 4, 40, [20, 33], 8, 2, 128, BF, S=40)
    for b, n in enumerate([20, 33]):
        x["v"][b, n - 1] = bad
        x["k"][b, n - 1] = bad if bad != bad else 0.5
    out, lse = _run_prefix(x)
    y = {n: t.clone() if t is not None else None for n, t in x.items()}
    for b, n in enumerate([20, 33]):
        y["v"][b, n - 1] = 0
        y["k"][b, n - 1] = 0
    want, want_lse, bound = ref.prefix_attention(y["q"], y["pk"], y["pv"], y["k"], y["v"], y["lengths"])
    _close(out[:, :3], want[:, :3], bound[:, :3], "earlier drafts")
    _lse_close(lse[:, :3], want_lse[:, :3])
    assert not bool(torch.isfinite(out[:, 3]).any())


def test_prefix_attention_page_ids_out_of_range_hold_nothing():
    x = _prefix_case(11, 3, 1, 33, [40, 40, 40], 4, 2, 64, BF, 8, S=40)
    x["table"][0, 1], x["table"][1, 0], x["table"][2] = -1, 10 ** 6, -7
    _check_prefix(x, "page ids")


def test_prefix_attention_strides_and_expanded_queries():
    """Operands cut out of one projection, head-major caches, one query for all."""
    g = _gen(12)
    B, T, Hq, H, D, P, S = 3, 2, 8, 2, 128, 70, 30
    qkv = torch.randn(B, T, (Hq + 2 * H) * D, generator=g).to(BF)
    kv = torch.randn(2, H, B, S, D, generator=g).to(BF)
    pkv = torch.randn(P, 2, H, D, generator=g).to(BF)
    lengths = torch.tensor([30, 2, 11], dtype=torch.int32)
    q = qkv[..., :Hq * D].view(B, T, Hq, D)
    k, v = kv[0].permute(1, 2, 0, 3), kv[1].permute(1, 2, 0, 3)
    want, want_lse, bound = ref.prefix_attention(q, pkv[:, 0], pkv[:, 1], k, v, lengths)
    c = kv.cuda()
    d = pkv.cuda()
    out, lse = serve.prefix_attention(qkv.cuda()[..., :Hq * D].view(B, T, Hq, D), d[:, 0], d[:, 1], c[0].permute(1, 2, 0, 3),
                                      c[1].permute(1, 2, 0, 3), lengths.cuda(), return_lse=True)
    _close(out, want, bound, "strides")
    _lse_close(lse, want_lse)
    one = torch.randn(1, 1, Hq, D, generator=g).to(BF)
    out = serve.prefix_attention(one.cuda().expand(B, 1, Hq, D), d[:, 0], d[:, 1], c[0].permute(1, 2, 0, 3),
                                 c[1].permute(1, 2, 0, 3), lengths.cuda())
    want, _, bound = ref.prefix_attention(one.expand(B, 1, Hq, D), pkv[:, 0], pkv[:, 1], k, v, lengths)
    _close(out, want, bound, "expanded")


def test_prefix_attention_gives_the_same_bits_again():
    x = _prefix_case(13, 9, 2, 3000, [2 + 11 * i for i in range(9)], 8, 2, 128, BF, 16)
    a, b = _run_prefix(x), _run_prefix(x)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def _cache_case(seed, B, H, C, D, lengths, dtype=BF, more=0):
    """A cache after `C + more` tokens, its positions out of order."""
    g = _gen(seed)
    positions = torch.rand(B, H, C + more, generator=g).argsort(-1)[..., :C].to(torch.int32).contiguous()
    weights = torch.exp(torch.randn(B, H, C, generator=g))
    weights[torch.rand(B, H, C, generator=g) < 0.2] = 0.0
    return dict(k=_randn(g, B, H, C, D, dtype=dtype), v=_randn(g, B, H, C, D, dtype=dtype), weights=weights,
                positions=positions, lengths=torch.tensor(lengths, dtype=torch.int32))


def _cuda_cache(x):
    return serve.BoundedCache(*(x[n].cuda() for n in ("k", "v", "weights", "positions", "lengths")))


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("B,T,C,Hq,H,D", [
    (1, 1, 1, 1, 1, 8), (2, 1, 33, 8, 2, 128), (3, 1, 300, 4, 4, 64), (2, 5, 129, 6, 2, 96), (1, 20, 260, 8, 1, 128),
    (2, 1, 1500, 7, 1, 256), (2, 2, 64, 40, 2, 80), (2, 33, 2100, 8, 2, 128), (1, 70, 1030, 4, 1, 256), (3, 40, 90, 2, 2, 64), (40, 4, 50, 8, 2, 64)])
def test_cache_attention(B, T, C, Hq, H, D, dtype):
    print("case", (B, T, C, Hq, H, D, dtype), flush=True)
    x = _cache_case(B + C + D, B, H, C, D, [C - (i * C) // (2 * B) for i in range(B)], dtype, more=9)
    # the first query token stands in the midst of the positions: some slots lie ahead of all, some of a few tokens
    pos = torch.tensor([(C + 9) * 2 // 3 + i for i in range(B)], dtype=torch.int32)
    q = _randn(_gen(T), B, T, Hq, D, dtype=dtype)
    want, want_w, bound = ref.cache_attention(q, pos=pos, **x)
    c = _cuda_cache(x)
    out = serve.cache_attention(q.cuda(), c, pos.cuda())
    _close(out, want, bound, "out")
    _close(c.weights, want_w, 2.0 ** -12 * (want_w - x["weights"].double()) + 2.0 ** -22 * want_w, "weights")


def test_cache_attention_unseen_slots_hold_anything():
    """Stale, empty and unused slots with NaN and infinities; a sequence that sees nothing."""
    x = _cache_case(21, 4, 2, 80, 64, [80, 50, 0, 80], more=5)
    pos = torch.tensor([60, 70, 50, -1], dtype=torch.int32)
    x["positions"][0, :, 7] = ref.NO_TOKEN
    x["positions"][1, 0, 3] = -5
    clean = {n: t.clone() for n, t in x.items()}
    for b in range(4):
        unseen = (torch.arange(80) >= x["lengths"][b]) | (x["positions"][b] > pos[b]) | (x["positions"][b] < 0)
        x["k"][b][unseen] = NAN
        x["v"][b][unseen] = INF
        clean["k"][b][unseen] = 0
        clean["v"][b][unseen] = 0
    q = _randn(_gen(1), 4, 1, 8, 64)
    want, want_w, bound = ref.cache_attention(q, pos=pos, **clean)
    c = _cuda_cache(x)
    out = serve.cache_attention(q.cuda(), c, pos.cuda())
    assert bool((out[2:] == 0).all())
    _close(out, want, bound, "out")
    _close(c.weights, want_w, 2.0 ** -12 * (want_w - x["weights"].double()) + 2.0 ** -22 * want_w, "weights")


def test_cache_attention_later_tokens_do_not_reach_earlier_ones():
    x = _cache_case(22, 2, 2, 50, 128, [50, 50])
    pos = torch.tensor([47, 47], dtype=torch.int32)
    last = x["positions"] == 49
    x["v"][last] = NAN
    clean = {n: t.clone() for n, t in x.items()}
    clean["v"][last] = 0
    q = _randn(_gen(2), 2, 3, 4, 128)
    want, want_w, bound = ref.cache_attention(q, pos=pos, **clean)
    c = _cuda_cache(x)
    out = serve.cache_attention(q.cuda(), c, pos.cuda())
    _close(out[:, :2], want[:, :2], bound[:, :2], "earlier tokens")
    assert bool(torch.isnan(out[:, 2]).all())
    _close(c.weights, want_w, 2.0 ** -12 * (want_w - x["weights"].double()) + 2.0 ** -22 * want_w, "weights")


@pytest.mark.parametrize("T,Hq,H,D,C", [(1, 2, 1, 64, 40), (3, 4, 2, 128, 700), (3, 4, 2, 128, 5000), (40, 2, 2, 128, 300), (70, 2, 1, 64, 150)])
def test_cache_attention_a_query_that_is_no_number_reaches_only_slots_it_sees(T, Hq, H, D, C):
    """One head's query of one token is NaN: its row, and the weights of the slots it sees, are; no others."""
    x = _cache_case(T + C, 2, H, C, D, [C, C - 3], more=6)
    pos = torch.tensor([C + 4 - T, C // 2], dtype=torch.int32)
    q = _randn(_gen(T), 2, T, Hq, D)
    clean = q.clone()
    bad = T // 3
    q[:, bad, Hq - 1] = NAN
    want, want_w, bound = ref.cache_attention(clean, pos=pos, **x)
    c = _cuda_cache(x)
    out = serve.cache_attention(q.cuda(), c, pos.cuda()).cpu()
    assert bool(torch.isnan(out[:, bad, Hq - 1]).all())
    out[:, bad, Hq - 1] = want[:, bad, Hq - 1].to(out.dtype)
    _close(out, want, bound, "other rows")
    there = torch.arange(C) < x["lengths"].view(-1, 1, 1)
    reached = there & (x["positions"] <= pos.view(-1, 1, 1) + bad) & (torch.arange(H).view(1, -1, 1) == H - 1)
    got = c.weights.cpu()
    assert bool((~there | (x["positions"] > pos.view(-1, 1, 1) + bad)).any())
    assert torch.equal(torch.isnan(got), reached)
    got[reached] = want_w[reached].to(got.dtype)
    _close(got, want_w, 2.0 ** -12 * (want_w - x["weights"].double()) + 2.0 ** -22 * want_w, "weights")


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("T,Hq,H,D,C", [(24, 4, 2, 128, 300), (40, 1, 1, 64, 150), (33, 4, 4, 256, 70), (9, 8, 2, 72, 129)])
def test_cache_attention_window_with_values_that_are_no_numbers(T, Hq, H, D, C, bad, dtype):
    """Many rows: the three last positions' values, and every unseen slot, hold `bad`."""
    x = _cache_case(T + D, 2, H, C, D, [C, C - 5], dtype, more=4)
    pos = torch.tensor([C + 4 - T, C - 10 - T], dtype=torch.int32)
    clean = {n: t.clone() for n, t in x.items()}
    first_bad = []
    for b in range(2):
        last = int(pos[b]) + T - 1
        unseen = (torch.arange(C) >= x["lengths"][b]) | (x["positions"][b] > last)
        late = ~unseen & (x["positions"][b] > last - 3)
        x["k"][b][unseen] = bad
        x["v"][b][unseen | late] = bad
        clean["k"][b][unseen] = 0
        clean["v"][b][unseen | late] = 0
        first_bad.append([T - 3 + int(3 - 1 - (last - x["positions"][b, h][late[h]]).max()) if late[h].any() else T
                          for h in range(H)])
    q = _randn(_gen(T), 2, T, Hq, D, dtype=dtype)
    want, want_w, bound = ref.cache_attention(q, pos=pos, **clean)
    c = _cuda_cache(x)
    out = serve.cache_attention(q.cuda(), c, pos.cuda()).cpu()
    for b in range(2):
        for h in range(H):
            heads, t = slice(h * (Hq // H), (h + 1) * (Hq // H)), first_bad[b][h]
            _close(out[b, :t, heads], want[b, :t, heads], bound[b, :t, heads], (b, h))
            assert not bool(torch.isfinite(out[b, t:, heads]).any())
    _close(c.weights, want_w, 2.0 ** -12 * (want_w - x["weights"].double()) + 2.0 ** -22 * want_w, "weights")


@pytest.mark.parametrize("B,H,C,D,lengths,pos,recent", [
    (1, 1, 1, 8, [0], [0], 1), (1, 1, 1, 8, [1], [5], 1), (2, 3, 40, 64, [40, 40], [49, 49], 8),
    (3, 2, 300, 128, [300, 17, 299], [320, 17, 299], 30), (2, 2, 64, 80, [64, 64], [40, -1], 0),
    (1, 2, 500, 256, [500], [520], 500), (2, 1, 33, 72, [33, 33], [60, 60], 10 ** 10),
    (1, 2, 9001, 8, [9001], [9010], 40)])
def test_cache_insert(B, H, C, D, lengths, pos, recent):
    x = _cache_case(C + D, B, H, C, D, lengths, more=20)
    if C > 30:
        x["weights"][0, 0, 11], x["weights"][0, 0, 5] = NAN, -0.0
    g = _gen(3)
    k_new, v_new = _randn(g, B, 1, H, D), _randn(g, B, 1, H, D)
    p = torch.tensor(pos, dtype=torch.int32)
    slots, new = ref.cache_insert(x["positions"], x["weights"], x["lengths"], p, recent)
    c = _cuda_cache(x)
    got, lengths_new = serve.cache_insert(c, k_new.cuda()[:, 0], v_new.cuda()[:, 0], p.cuda(), recent)
    assert torch.equal(got.cpu(), slots) and torch.equal(lengths_new.cpu(), new)
    assert torch.equal(c.lengths.cpu(), x["lengths"])
    for b in range(B):
        for h in range(H):
            i = int(slots[b, h])
            if i >= 0:
                x["k"][b, h, i], x["v"][b, h, i] = k_new[b, 0, h], v_new[b, 0, h]
                x["weights"][b, h, i], x["positions"][b, h, i] = 0.0, pos[b]
    for n in ("k", "v", "positions"):
        assert torch.equal(getattr(c, n).cpu(), x[n]), n
    assert np.array_equal(c.weights.cpu().numpy(), x["weights"].numpy(), equal_nan=True)


def test_cache_insert_takes_stale_slots_first_and_fills_by_weight():
    """Ten tokens one after another against the definition, the cache's own state carried along."""
    x = _cache_case(31, 2, 2, 24, 64, [20, 24], more=0)
    x["positions"][1, 0, 7] = 90   # refused drafts
    x["positions"][1, 1, 2] = ref.NO_TOKEN
    c = _cuda_cache(x)
    positions, weights, lengths = x["positions"].clone(), x["weights"].clone(), x["lengths"].clone()
    for step in range(10):
        p = torch.tensor([24 + step, 30 + step], dtype=torch.int32)
        slots, new = ref.cache_insert(positions, weights, lengths, p, 4)
        row = torch.full((2, 2, 64), float(step)).to(BF).cuda()
        got, grown = serve.cache_insert(c, row, row, p.cuda(), 4)
        c.set_lengths(grown)
        assert torch.equal(got.cpu(), slots) and torch.equal(grown.cpu(), new), step
        for b in range(2):
            for h in range(2):
                positions[b, h, slots[b, h]] = p[b]
                weights[b, h, slots[b, h]] = 0.0
        lengths = new
    assert torch.equal(c.positions.cpu(), positions)


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("B,H,C,D,lengths,budget,recent,slots", [
    (1, 1, 1, 8, [1], 1, 0, 1), (2, 2, 100, 64, [100, 60], 40, 10, 40), (2, 1, 2500, 128, [2500, 1030], 1025, 1025, 1100),
    (3, 2, 300, 80, [300, 20, 0], 64, 0, 70), (1, 3, 5000, 256, [4999], 700, 33, 700), (1, 2, 70001, 8, [70000], 9000, 100, 9000),
    (1, 1, 12000, 8, [12000], 50, 0, 50)])
def test_cache_compact(B, H, C, D, lengths, budget, recent, slots, dtype):
    x = _cache_case(C + D, B, H, C, D, lengths, dtype, more=7)
    if C >= 100:
        x["weights"][0, 0, 3:9] = torch.tensor([NAN, INF, -INF, 0.0, -0.0, 0.0])
        x["positions"][0, 0, 20] = ref.NO_TOKEN
        x["positions"][0, 0, 21] = -1
        x["weights"] = (x["weights"] * 4).round() / 4   # many equal weights
    pos = torch.tensor([C + 2 - i for i in range(B)], dtype=torch.int32)
    want = ref.cache_compact(x["positions"], x["weights"], x["lengths"], pos, budget, recent)
    c = _cuda_cache(x)
    cut, kept = serve.cache_compact(c, pos.cuda(), budget, recent, slots=slots)
    kept = kept.cpu()
    assert kept.shape == (B, H, slots) and torch.equal(kept[..., :budget], want) and bool((kept[..., budget:] == -1).all())
    assert torch.equal(cut.lengths.cpu(), x["lengths"].clamp(max=budget))
    there, at = kept >= 0, kept.clamp(min=0).long()
    rows = at.unsqueeze(-1).expand(B, H, slots, D)
    for n in ("k", "v"):
        assert torch.equal(getattr(cut, n).cpu(), torch.where(there.unsqueeze(-1), x[n].gather(2, rows), 0)), n
    assert torch.equal(cut.positions.cpu(), torch.where(there, x["positions"].gather(2, at), ref.NO_TOKEN))
    assert np.array_equal(cut.weights.cpu().numpy(), torch.where(there, x["weights"].gather(2, at), 0.0).numpy(), equal_nan=True)
    for n in ("k", "v", "positions", "lengths"):
        assert torch.equal(getattr(c, n).cpu(), x[n]), "the cache itself is left alone"


def _verify_case(seed, B, G, V, dtype, spread=0.5):
    g = _gen(seed)
    logits = 2.0 * torch.randn(B, G + 1, V, generator=g)
    target = torch.softmax(logits, -1)
    draft = torch.softmax(logits[:, :G] + spread * torch.randn(B, G, V, generator=g), -1)
    tokens = torch.multinomial(draft.reshape(-1, V), 1, generator=g).view(B, G) if G else torch.zeros(B, 0, dtype=torch.int64)
    return dict(draft_tokens=tokens, target=target.to(dtype), uniforms=torch.rand(B, G + 1, generator=g), draft=draft.to(dtype))


def _check_verify(x, counts=None):
    want = ref.verify_drafts(counts=counts, **x)
    draft = x["draft"].cuda() if x["draft"] is not None else None
    got = serve.verify_drafts(x["draft_tokens"].cuda(), x["target"].cuda(), x["uniforms"].cuda(), draft,
                              counts=counts.cuda() if counts is not None else None)
    assert got[0].dtype == x["draft_tokens"].dtype
    assert torch.equal(got[1].cpu(), want[1])
    assert torch.equal(got[0].cpu(), want[0])
    return want


@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("B,G,V", [(1, 1, 1), (3, 0, 7), (8, 3, 33), (4, 5, 1000), (6, 4, 5003), (2, 7, 40000), (1, 2, 600011)])
def test_verify_drafts(B, G, V, dtype):
    print("case", (B, G, V, dtype), flush=True)
    x = _verify_case(B + G + V, B, G, V, dtype)
    _check_verify(x)
    x["draft_tokens"] = x["draft_tokens"].to(torch.int32)
    _check_verify(x, torch.tensor([(3 * i - 1) % (G + 3) - 1 for i in range(B)], dtype=torch.int32))
    x["draft"] = None
    _check_verify(x)


def test_verify_drafts_takes_and_refuses():
    """Uniforms at their ends: all drafts taken, none taken."""
    x = _verify_case(41, 6, 4, 301, F32)
    x["uniforms"][:3, :4] = 0.0
    x["uniforms"][3:, :4] = 1.0 - 2.0 ** -24
    x["uniforms"][::2, 4], x["uniforms"][1::2, 4] = 0.0, 1.0 - 2.0 ** -24
    _, accepted = _check_verify(x)
    assert accepted[:3].tolist() == [4, 4, 4]


def test_verify_drafts_edges():
    """Tokens outside the vocabulary, equal distributions (nothing left of
    p - q), rows without any probability, values that are no probabilities."""
    x = _verify_case(42, 7, 3, 130, F32)
    x["draft_tokens"][0, 1], x["draft_tokens"][1, 0] = 130, -1
    x["draft"][2] = x["target"][2, :3]
    x["uniforms"][2, :3] = 1.0 - 2.0 ** -24
    x["target"][2, 1] *= 0.5
    x["target"][3] = 0.0
    x["target"][4, :, ::2], x["target"][4, :, 1::7] = NAN, -1.0
    x["target"][5, :, 5] = INF
    x["draft"][6] = NAN
    tokens, accepted = _check_verify(x)
    assert tokens[3].tolist() == [-1, -1, -1, -1] and accepted[3] == 0


def test_verify_drafts_strided_probabilities():
    x = _verify_case(43, 4, 3, 97, BF)
    wide = torch.zeros(4, 9, 101, dtype=BF)
    wide[:, 1:5, 2:99] = x["target"]
    other = torch.zeros(3, 4, 97, dtype=BF)
    other.copy_(x["draft"].transpose(0, 1))
    want = ref.verify_drafts(**x)
    got = serve.verify_drafts(x["draft_tokens"].cuda(), wide.cuda()[:, 1:5, 2:99], x["uniforms"].cuda(),
                              other.cuda().transpose(0, 1))
    assert torch.equal(got[0].cpu(), want[0]) and torch.equal(got[1].cpu(), want[1])


def test_verify_drafts_distribution():
    """What is emitted first is distributed as the target, whatever the drafter."""
    V, n = 6, 40000
    target = torch.tensor([0.3, 0.05, 0.25, 0.1, 0.2, 0.1])
    draft = torch.tensor([0.1, 0.4, 0.1, 0.2, 0.15, 0.05])
    g = _gen(44)
    tokens = torch.multinomial(draft.expand(n, V), 1, generator=g).to(torch.int32)
    out, _ = serve.verify_drafts(tokens.cuda(), target.expand(n, 2, V).cuda(), torch.rand(n, 2, generator=g).cuda(),
                                 draft.expand(n, 1, V).cuda())
    share = torch.bincount(out[:, 0].cpu().long(), minlength=V).double() / n
    # five standard deviations of a share of at most 0.3 among 40000
    assert float((share - target).abs().max()) < 5 * (0.3 * 0.7 / n) ** 0.5


def test_operators_run_on_the_given_stream():
    """Inputs made on one side stream, operators on it by `stream`, another stream current."""
    side = torch.cuda.Stream()
    x = _prefix_case(51, 3, 1, 600, [5, 60, 128], 8, 2, 128, BF, 16)
    y = _cache_case(52, 2, 2, 90, 64, [90, 45])
    q, pos = _randn(_gen(5), 2, 1, 4, 64), torch.tensor([95, 60], dtype=torch.int32)
    v = _verify_case(53, 3, 2, 500, F32)
    cut_want = ref.cache_compact(y["positions"], y["weights"], y["lengths"], pos, 30, 5)
    with torch.cuda.stream(side):
        big = torch.randn(4096, 4096, device="cuda")
        for _ in range(10):
            big = big @ big * 1e-3   # the side stream is busy when the operators are enqueued
        c = {n: t.cuda() if t is not None else None for n, t in x.items()}
        cache = _cuda_cache(y)
        qc, pc = q.cuda(), pos.cuda()
        vc = {n: t.cuda() for n, t in v.items()}
    cut, kept = serve.cache_compact(cache, pc, 30, 5, stream=side)
    out, lse = serve.prefix_attention(c["q"], c["pk"], c["pv"], c["k"], c["v"], c["lengths"], block_table=c["table"],
                                      return_lse=True, stream=side)
    att = serve.cache_attention(qc, cache, pc, stream=side)
    tokens, accepted = serve.verify_drafts(vc["draft_tokens"], vc["target"], vc["uniforms"], vc["draft"], stream=side)
    side.synchronize()
    want, want_lse, bound = ref.prefix_attention(x["q"], x["pk"], x["pv"], x["k"], x["v"], x["lengths"], x["table"])
    _close(out, want, bound, "prefix")
    _lse_close(lse, want_lse)
    want, _, bound = ref.cache_attention(q, pos=pos, **y)
    _close(att, want, bound, "cache")
    assert torch.equal(kept.cpu(), cut_want)
    assert torch.equal(tokens.cpu(), ref.verify_drafts(**v)[0])


def test_operators_in_a_graph():
    """Captured once, replayed several times with other inputs in place and
    eager work between the replays; each replay against the eager result."""
    x = _prefix_case(61, 3, 2, 700, [5, 60, 128], 8, 2, 128, BF, 16)
    c = {n: t.cuda() if t is not None else None for n, t in x.items()}
    y = _cache_case(62, 2, 2, 90, 64, [90, 90])
    cache, q = _cuda_cache(y), _randn(_gen(6), 2, 1, 4, 64).cuda()
    pos = torch.tensor([95, 96], dtype=torch.int32).cuda()
    row = _randn(_gen(7), 2, 2, 64).cuda()
    v = {n: t.cuda() for n, t in _verify_case(63, 3, 2, 5000, F32).items()}

    def step():
        a = serve.prefix_attention(c["q"], c["pk"], c["pv"], c["k"], c["v"], c["lengths"], block_table=c["table"])
        slots, _ = serve.cache_insert(cache, row, row, pos, 8)
        b = serve.cache_attention(q, cache, pos)
        cut, kept = serve.cache_compact(cache, pos, 40, 8)
        d = serve.verify_drafts(v["draft_tokens"], v["target"], v["uniforms"], v["draft"])
        return a, slots, b, cut.k, kept, d[0], d[1]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()
    for i in range(4):
        c["q"].copy_(torch.randn(c["q"].shape, generator=_gen(70 + i)).to(BF))
        v["uniforms"].copy_(torch.rand(v["uniforms"].shape, generator=_gen(80 + i)))
        pos.add_(1)
        before = cache.weights.clone(), cache.positions.clone(), cache.k.clone(), cache.v.clone()
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in held]
        state = cache.weights.clone(), cache.positions.clone()
        for t, old in zip((cache.weights, cache.positions, cache.k, cache.v), before):
            t.copy_(old)
        for a, b in zip(got, step()):
            assert torch.equal(a, b)
        assert torch.equal(cache.weights, state[0]) and torch.equal(cache.positions, state[1])
        torch.cuda.synchronize()


def test_empty_batches():
    z = torch.zeros
    out, lse = serve.prefix_attention(z(0, 1, 4, 64, dtype=BF, device="cuda"), z(9, 2, 64, dtype=BF, device="cuda"),
                                      z(9, 2, 64, dtype=BF, device="cuda"), z(0, 5, 2, 64, dtype=BF, device="cuda"),
                                      z(0, 5, 2, 64, dtype=BF, device="cuda"), z(0, dtype=torch.int32, device="cuda"),
                                      return_lse=True)
    assert out.shape == (0, 1, 4, 64) and lse.shape == (0, 1, 4)
    cache = serve.BoundedCache.empty(0, 2, 8, 64)
    none = z(0, dtype=torch.int32, device="cuda")
    assert serve.cache_attention(z(0, 1, 4, 64, dtype=BF, device="cuda"), cache, none).shape == (0, 1, 4, 64)
    slots, _ = serve.cache_insert(cache, z(0, 2, 64, dtype=BF, device="cuda"), z(0, 2, 64, dtype=BF, device="cuda"), none, 1)
    assert slots.shape == (0, 2)
    assert serve.cache_compact(cache, none, 4, 1)[1].shape == (0, 2, 4)
    tokens, accepted = serve.verify_drafts(z(0, 3, dtype=torch.int32, device="cuda"), z(0, 4, 50, device="cuda"),
                                           z(0, 4, device="cuda"))
    assert tokens.shape == (0, 4) and accepted.shape == (0,)


def test_refusals():
    z = torch.zeros
    q, k = z(2, 1, 4, 64, dtype=BF, device="cuda"), z(2, 8, 2, 64, dtype=BF, device="cuda")
    p, n = z(16, 2, 64, dtype=BF, device="cuda"), z(2, dtype=torch.int32, device="cuda")
    att = serve.prefix_attention
    with pytest.raises(ValueError):
        att(q.cpu(), p, p, k, k, n)
    with pytest.raises(TypeError):
        att(q.float(), p, p, k, k, n)
    with pytest.raises(TypeError):
        att(q, p.half(), p, k, k, n)
    with pytest.raises(TypeError):
        att(q, p, p, k, k, n.long())
    with pytest.raises(ValueError):
        att(q, p, p, k, k, n[:1])
    with pytest.raises(ValueError):
        att(q, p, p, k, k[:, :4], n)
    with pytest.raises(ValueError):
        att(q, p, p.transpose(0, 1).contiguous().transpose(0, 1), k, k, n)
    with pytest.raises(ValueError):
        att(q, p, p, k.transpose(2, 3).contiguous().transpose(2, 3), k.transpose(2, 3).contiguous().transpose(2, 3), n)
    with pytest.raises(RuntimeError):
        att(z(2, 1, 3, 64, dtype=BF, device="cuda"), p, p, k, k, n)          # 3 heads over 2 key heads
    with pytest.raises(RuntimeError):
        att(z(2, 1, 4, 60, dtype=BF, device="cuda"), p[..., :60].contiguous(), p[..., :60].contiguous(),
            k[..., :60].contiguous(), k[..., :60].contiguous(), n)
    flat = z(2 * 8 * 2 * 64 + 8, dtype=BF, device="cuda")
    off = flat[1:1 + 2 * 8 * 2 * 64].view(2, 8, 2, 64)
    with pytest.raises(RuntimeError):
        att(q, p, p, off, off, n)                                             # not 16-byte aligned
    with pytest.raises(ValueError):
        att(q, p, p, k, k, n, block_table=z(3, 1, dtype=torch.int32, device="cuda"))
    cache = serve.BoundedCache.empty(2, 2, 8, 64)
    with pytest.raises(TypeError):
        serve.BoundedCache(cache.k, cache.v, cache.weights.half(), cache.positions, cache.lengths)
    with pytest.raises(ValueError):
        serve.BoundedCache(cache.k, cache.v, cache.weights[:1], cache.positions, cache.lengths)
    with pytest.raises(AttributeError):
        cache.lengths = n
    with pytest.raises(ValueError):
        serve.cache_attention(z(3, 1, 4, 64, dtype=BF, device="cuda"), cache, n)
    with pytest.raises(ValueError):
        serve.cache_insert(cache, q[:, 0], q[:, 0], n, 1)                     # 4 heads, the cache has 2
    with pytest.raises(RuntimeError):
        serve.cache_insert(cache, k[:, 0], k[:, 0], n, -1)
    with pytest.raises(RuntimeError):
        serve.cache_compact(cache, n, 4, 5)
    with pytest.raises(RuntimeError):
        serve.cache_compact(cache, n, 4, 1, slots=3)
    with pytest.raises(ValueError):
        serve.verify_drafts(z(2, 3, dtype=torch.int32, device="cuda"), z(2, 3, 50, device="cuda"), z(2, 4, device="cuda"))
    with pytest.raises(TypeError):
        serve.verify_drafts(z(2, 3, dtype=torch.int16, device="cuda"), z(2, 4, 50, device="cuda"), z(2, 4, device="cuda"))
    with pytest.raises(TypeError):
        serve.verify_drafts(z(2, 3, dtype=torch.int32, device="cuda"), z(2, 4, 50, device="cuda"), z(2, 4, device="cuda"),
                            z(2, 3, 50, dtype=BF, device="cuda"))


@pytest.mark.parametrize("C,used,recent", [(24, 24, 4), (40, 24, 4), (16, 16, 16)])
def test_refused_drafts_are_not_seen_again(C, used, recent):
    """Rounds of drafts into full and not full caches, a full one's in slots of
    descending index, all or some of them refused and forgotten: after each
    insertion the attention is that over the tokens that were kept, held
    beside the cache by their positions."""
    B, H, D, drafts = 2, 2, 64, 4
    x = _cache_case(41 + C, B, H, C, D, [used] * B)
    for b in range(B):
        for h in range(H):
            x["positions"][b, h, :used] = torch.randperm(used, generator=_gen(2 * b + h))
    x["positions"][:, :, used:] = ref.NO_TOKEN
    x["weights"] = torch.arange(C, 0, -1, dtype=torch.float32).expand(B, H, C).contiguous()   # the last slot is the lightest
    c = _cuda_cache(x)
    held = {(b, h): {int(x["positions"][b, h, i]): (i, x["k"][b, h, i], x["v"][b, h, i]) for i in range(used)}
            for b in range(B) for h in range(H)}
    g, nxt = _gen(5), [used] * B
    for turn in range(8):
        for step in range(drafts):
            pos = torch.tensor([n + step for n in nxt], dtype=torch.int32)
            k_new, v_new = _randn(g, B, H, D), _randn(g, B, H, D)
            slots, lengths = serve.cache_insert(c, k_new.cuda(), v_new.cuda(), pos.cuda(), recent)
            c.set_lengths(lengths)
            for (b, h), tokens in held.items():
                for p in [p for p, t in tokens.items() if t[0] == int(slots[b, h])]:
                    del tokens[p]
                assert int(pos[b]) not in tokens
                tokens[int(pos[b])] = (int(slots[b, h]), k_new[b, h], v_new[b, h])
            q = _randn(g, B, 1, 2 * H, D)
            out = serve.cache_attention(q.cuda(), c, pos.cuda()).cpu()
            for b in range(B):
                for head in range(2 * H):
                    tokens = held[b, head // 2].values()
                    want, _, _, bound = ref.attend(q[b, 0, head], torch.stack([t[1] for t in tokens]),
                                                   torch.stack([t[2] for t in tokens]), D ** -0.5)
                    _close(out[b, 0, head], want, bound, (turn, step, b, head))
            # weights as the caller likes them: the least in the last slot, so that evictions go downwards
            c.weights.copy_(x["weights"])
        kept = [(turn * 3 + b) % drafts for b in range(B)]   # none, some, all but one
        nxt = [n + k for n, k in zip(nxt, kept)]
        c.forget(torch.tensor(nxt, dtype=torch.int32, device="cuda"))
        for (b, h), tokens in held.items():
            for p in [p for p in tokens if p >= nxt[b]]:
                del tokens[p]
            live = c.positions[b, h, :int(c.lengths[b])].cpu()
            assert sorted(tokens) == sorted(live[live != ref.NO_TOKEN].tolist())


def test_forget():
    """Other sequences, a negative position, the arguments."""
    x = _cache_case(43, 3, 2, 30, 64, [30, 20, 30])
    c = _cuda_cache(x)
    c.forget(torch.tensor([10, 25, -1], dtype=torch.int32, device="cuda"))
    want = x["positions"].clone()
    for b, n in ((0, 10), (1, 25)):
        want[b][want[b] >= n] = ref.NO_TOKEN
    assert torch.equal(c.positions.cpu(), want)
    for n in ("k", "v", "weights", "lengths"):
        assert torch.equal(getattr(c, n).cpu(), x[n]), n
    with pytest.raises(TypeError):
        c.forget(torch.tensor([10, 25, -1], device="cuda"))
    with pytest.raises(TypeError):
        c.forget(10)
    with pytest.raises(ValueError):
        c.forget(torch.tensor([10, 25], dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        c.forget(torch.tensor([10, 25, 3], dtype=torch.int32))


@pytest.mark.parametrize("D,token", [(64, 1 << 25), (64, 34_700_000), (128, 1 << 25), (128, 71_600_000), (72, (1 << 27) - 8)])
def test_rows_far_apart(D, token):
    """Many rows over keys whose rows lie `token` elements apart: at the most
    that 128-row tiles take, where a tile's lane distance (124 or 60 rows)
    passes 2^32 elements, and at the most that any call takes."""
    n = min(2 * 8192 // 64 if D == 64 else 8192 // 64, 6_000_000_000 // token)   # keys: 6e9 elements at most
    H = 2
    if torch.cuda.mem_get_info()[0] < 2 * n * token + (8 << 30):
        pytest.skip("needs %d GB of device memory" % (2 * n * token + (8 << 30) >> 30))
    assert token <= 1 << 25 or n > 40
    flat = torch.empty((n - 1) * token + 2 * H * D + 64, dtype=BF, device="cuda")
    far_k, far_v = (flat[i * H * D:].as_strided((n, H, D), (token, D, 1)) for i in range(2))
    g = _gen(D)
    pk, pv = _randn(g, n, H, D), _randn(g, n, H, D)
    far_k.copy_(pk), far_v.copy_(pv)
    q, k, v = _randn(g, 10, 1, 4, D), _randn(g, 10, 3, H, D), _randn(g, 10, 3, H, D)   # 20 rows of a key head
    lengths = torch.full((10,), 3, dtype=torch.int32)
    out, lse = serve.prefix_attention(q.cuda(), far_k, far_v, k.cuda(), v.cuda(), lengths.cuda(), return_lse=True)
    want, want_lse, bound = ref.prefix_attention(q, pk, pv, k, v, lengths)
    _close(out, want, bound, "prefix")
    _lse_close(lse, want_lse)
    # the same rows as a cache's slots, under a window of 40 query tokens
    x = dict(k=pk.transpose(0, 1)[None], v=pv.transpose(0, 1)[None], weights=torch.zeros(1, H, n),
             positions=torch.arange(n, dtype=torch.int32).expand(1, H, n).contiguous(),
             lengths=torch.tensor([n], dtype=torch.int32))
    pos = torch.tensor([n - 40], dtype=torch.int32)
    cache = serve.BoundedCache(far_k.transpose(0, 1)[None], far_v.transpose(0, 1)[None],
                               *(x[name].cuda() for name in ("weights", "positions", "lengths")))
    q = _randn(g, 1, 40, 2, D)
    want, want_w, bound = ref.cache_attention(q, pos=pos, **x)
    _close(serve.cache_attention(q.cuda(), cache, pos.cuda()), want, bound, "window")
    _close(cache.weights, want_w, 2.0 ** -12 * want_w + 2.0 ** -22 * want_w, "weights")


@pytest.mark.parametrize("first", [-3, -39, -(1 << 31)])
def test_cache_attention_window_from_before_the_first_position(first):
    """Many rows from a negative position on: tokens before position 0 see
    nothing; a value that is no number at position 5 reaches the tokens from
    there on, those of empty slots none."""
    T, C = 40, 150
    x = _cache_case(4, 1, 1, C, 64, [C])
    x["positions"][0, 0] = torch.arange(C, dtype=torch.int32)
    x["positions"][0, 0, 20:140] = ref.NO_TOKEN
    x["v"][0, 0, 20:140] = NAN
    clean = {n: t.clone() for n, t in x.items()}
    clean["v"][0, 0, 20:140] = 0
    x["v"][0, 0, 5] = NAN
    pos = torch.tensor([first], dtype=torch.int32)
    q = _randn(_gen(2), 1, T, 1, 64)
    c = _cuda_cache(x)
    out = serve.cache_attention(q.cuda(), c, pos.cuda()).cpu()
    at = first + torch.arange(T)
    assert torch.equal(torch.isnan(out).any(-1)[0, :, 0], at >= 5)
    assert bool((out[0, at < 0] == 0).all())
    want, want_w, bound = ref.cache_attention(q, pos=pos, **clean)
    _close(out[:, at < 5], want[:, at < 5], bound[:, at < 5], "tokens before the value")
    _close(c.weights, want_w, 2.0 ** -12 * (want_w - x["weights"].double()) + 2.0 ** -22 * want_w, "weights")


@pytest.mark.parametrize("T", [1, 40, 400])
def test_attention_in_the_place_of_its_queries(T):
    """out=q, few rows and many (whose weights are taken from q once more):
    the same bits as into another tensor."""
    x = _cache_case(3, 2, 2, 300, 128, [300, 290], more=9)
    pos = torch.tensor([250, 260], dtype=torch.int32).cuda()
    q = _randn(_gen(1), 2, T, 4, 128).cuda()
    a, b = _cuda_cache(x), _cuda_cache(x)
    out = serve.cache_attention(q, a, pos)
    same = q.clone()
    assert serve.cache_attention(same, b, pos, out=same).data_ptr() == same.data_ptr()
    assert torch.equal(out, same) and torch.equal(a.weights, b.weights)
    y = {n: t.cuda() if t is not None else None for n, t in _prefix_case(2, 2, T, 99, [T, T + 4], 4, 2, 128, BF).items()}
    out = serve.prefix_attention(y["q"], y["pk"], y["pv"], y["k"], y["v"], y["lengths"])
    serve.prefix_attention(y["q"], y["pk"], y["pv"], y["k"], y["v"], y["lengths"], out=y["q"])
    assert torch.equal(out, y["q"])


@pytest.mark.parametrize("how", ["copied", "pickled"])
def test_a_copy_of_a_cache_has_its_own_memory(how):
    a = _cuda_cache(_cache_case(4, 2, 2, 20, 64, [20, 11]))
    b = copy.deepcopy(a) if how == "copied" else pickle.loads(pickle.dumps(a))
    names = ("k", "v", "weights", "positions", "lengths")
    before = [getattr(a, n).clone() for n in names]
    row, pos = _randn(_gen(1), 2, 2, 64).cuda(), torch.tensor([30, 31], dtype=torch.int32, device="cuda")
    slots, _ = serve.cache_insert(b, row, row, pos, 2)
    serve.cache_attention(row[:, None], b, pos)
    for n, t in zip(names, before):
        assert torch.equal(getattr(a, n), t), n
    for i in range(2):
        for h in range(2):
            assert torch.equal(b.k[i, h, int(slots[i, h])], row[i, h]) and int(b.positions[i, h, int(slots[i, h])]) == 30 + i
    assert bool((b.weights != before[2]).any())


def test_a_cache_whose_tensors_get_other_memory():
    """set_, resize_: the next call uses the memory there is, or refuses its shape."""
    x = _cache_case(5, 2, 2, 40, 64, [40, 33])
    a, b = _cuda_cache(x), _cuda_cache(x)
    held = [getattr(a, n).untyped_storage() for n in ("k", "v", "weights", "positions")]
    for n in ("k", "v", "weights", "positions"):
        t = getattr(a, n)
        t.set_(t.clone())
    old = torch.empty(0, device="cuda").set_(held[2], 0, (2, 2, 40), (80, 40, 1)).clone()
    q, pos = _randn(_gen(1), 2, 1, 4, 64).cuda(), torch.tensor([35, 31], dtype=torch.int32, device="cuda")
    assert torch.equal(serve.cache_attention(q, a, pos), serve.cache_attention(q, b, pos))
    assert torch.equal(a.weights, b.weights) and bool((a.weights != x["weights"].cuda()).any())
    assert torch.equal(torch.empty(0, device="cuda").set_(held[2], 0, (2, 2, 40), (80, 40, 1)), old)
    a.k.resize_(2, 2, 20, 64)
    for call in (lambda: serve.cache_attention(q, a, pos), lambda: serve.cache_compact(a, pos, 4, 1),
                 lambda: serve.cache_insert(a, q[:, 0, :2], q[:, 0, :2], pos, 1)):
        with pytest.raises(ValueError):
            call()


def test_gradients_are_refused():
    """Each floating operand that requires a gradient, unless gradients are off."""
    x = {n: t.cuda() if t is not None else None for n, t in _prefix_case(1, 2, 1, 9, [3, 4], 4, 2, 64, BF).items()}
    y = _cache_case(6, 2, 2, 20, 64, [20, 20])
    cache, pos = _cuda_cache(y), torch.tensor([30, 30], dtype=torch.int32, device="cuda")
    q, row = _randn(_gen(2), 2, 1, 4, 64).cuda(), _randn(_gen(3), 2, 2, 64).cuda()
    tokens, target, uniforms = torch.zeros(2, 3, dtype=torch.int64, device="cuda"), torch.rand(2, 4, 50, device="cuda"), \
        torch.rand(2, 4, device="cuda")
    draft = target[:, :3].clone()
    calls = [(serve.prefix_attention, [x[n] for n in ("q", "pk", "pv", "k", "v", "lengths")], range(5)),
             (serve.cache_attention, [q, cache, pos], [0]),
             (serve.cache_insert, [cache, row, row.clone(), pos, 2], [1, 2]),
             (serve.verify_drafts, [tokens, target, uniforms, draft], [1, 2, 3]),
             (serve.BoundedCache, [y[n].cuda() for n in ("k", "v", "weights", "positions", "lengths")], range(3))]
    for call, args, floats in calls:
        call(*args)
        for i in floats:
            some = list(args)
            some[i] = args[i].clone().requires_grad_()
            with pytest.raises(ValueError, match="gradient"):
                call(*some)
            with torch.no_grad():
                call(*some)
    held = _cuda_cache(y)
    held.k.requires_grad_()
    for call in (lambda: serve.cache_attention(q, held, pos), lambda: serve.cache_compact(held, pos, 4, 1)):
        with pytest.raises(ValueError, match="gradient"):
            call()
        with torch.inference_mode():
            call()


def test_writes_in_place_are_counted():
    """The versions of what a call writes grow, those of what it reads do not; inference tensors have none."""
    c = _cuda_cache(_cache_case(7, 1, 2, 20, 64, [20]))
    names = ("k", "v", "weights", "positions", "lengths")
    version = lambda: [getattr(c, n)._version for n in names]   # noqa: E731
    row, q = _randn(_gen(1), 1, 2, 64).cuda(), _randn(_gen(2), 1, 1, 4, 64).cuda()
    pos, out = torch.tensor([30], dtype=torch.int32, device="cuda"), torch.empty(1, 1, 4, 64, dtype=BF, device="cuda")
    old = version()
    serve.cache_insert(c, row, row, pos, 2)
    assert [new > o for new, o in zip(version(), old)] == [True, True, True, True, False]
    old, old_out = version(), out._version
    serve.cache_attention(q, c, pos, out=out)
    assert [new > o for new, o in zip(version(), old)] == [False, False, True, False, False] and out._version > old_out
    old = version()
    serve.cache_compact(c, pos, 5, 1)
    assert version() == old and q._version == row._version == pos._version == 0
    old_out = out._version
    serve.prefix_attention(q, row.transpose(0, 1).expand(2, 2, 64).contiguous(), row.transpose(0, 1).expand(2, 2, 64).contiguous(),
                           row[:, None], row[:, None], pos, out=out)
    assert out._version > old_out
    with torch.inference_mode():
        other = _cuda_cache(_cache_case(7, 1, 2, 20, 64, [20]))
    serve.cache_insert(other, row, row, pos, 2)
    serve.cache_attention(q, other, pos)


@pytest.mark.parametrize("yes,no", [(True, False), (1, 0), (np.bool_(True), np.bool_(False)), ("yes", None)])
def test_return_lse_is_any_truth_value(yes, no):
    x = {n: t.cuda() if t is not None else None for n, t in _prefix_case(1, 2, 1, 9, [3, 4], 4, 2, 64, BF).items()}
    args = [x[n] for n in ("q", "pk", "pv", "k", "v", "lengths")]
    out, lse = serve.prefix_attention(*args, return_lse=yes)
    assert lse.shape == (2, 1, 4)
    assert torch.equal(serve.prefix_attention(*args, return_lse=no), out)
    with pytest.raises(ValueError):   # an array of two has no truth value
        serve.prefix_attention(*args, return_lse=np.array([True, False]))


def test_expanded_caches_are_read_and_not_written():
    """Heads that share one key tensor: attention and compaction as of a cache
    of copies, insertion refused; head-last and interleaved caches are written."""
    x = _cache_case(8, 2, 1, 30, 64, [30, 25])
    c = {n: t.cuda() for n, t in x.items()}
    both = {n: c[n].expand(2, 4, 30).contiguous() for n in ("weights", "positions")}
    shared = serve.BoundedCache(c["k"].expand(2, 4, 30, 64), c["v"].expand(2, 4, 30, 64), both["weights"], both["positions"],
                                c["lengths"])
    copies = serve.BoundedCache(c["k"].repeat(1, 4, 1, 1), c["v"].repeat(1, 4, 1, 1), both["weights"].clone(),
                                both["positions"], c["lengths"])
    q, pos = _randn(_gen(1), 2, 1, 8, 64).cuda(), torch.tensor([28, 29], dtype=torch.int32, device="cuda")
    assert torch.equal(serve.cache_attention(q, shared, pos), serve.cache_attention(q, copies, pos))
    assert torch.equal(shared.weights, copies.weights)
    a, b = serve.cache_compact(shared, pos, 9, 2), serve.cache_compact(copies, pos, 9, 2)
    assert torch.equal(a[1], b[1]) and torch.equal(a[0].k, b[0].k)
    row = _randn(_gen(2), 2, 4, 64).cuda()
    before = c["k"].clone()
    with pytest.raises(RuntimeError, match="share memory"):
        serve.cache_insert(shared, row, row, pos, 2)
    assert torch.equal(c["k"], before)
    slots, _ = serve.cache_insert(copies, row, row, pos, 2)
    for layout in ("slots before heads", "keys beside values"):
        if layout == "slots before heads":
            k, v = (t.repeat(1, 4, 1, 1).transpose(1, 2).contiguous().transpose(1, 2) for t in (c["k"], c["v"]))
        else:
            k, v = torch.stack([c["k"].repeat(1, 4, 1, 1), c["v"].repeat(1, 4, 1, 1)], 3).unbind(3)
        other = serve.BoundedCache(k, v, shared.weights.clone(), c["positions"].expand(2, 4, 30).contiguous(), c["lengths"])
        got, _ = serve.cache_insert(other, row, row, pos, 2)
        assert torch.equal(got, slots) and torch.equal(other.k, copies.k) and torch.equal(other.v, copies.v)


def test_cache_compact_within_one_allocation():
    """Old and new slots behind each other in one allocation's rows."""
    import ctypes

    from huffman_decode_df11_amd import _lib
    B, H, C, N, D = 2, 2, 50, 20, 64
    x = _cache_case(9, B, H, C, D, [50, 41], more=5)
    pool = torch.zeros(2, B, H, C + N, D, dtype=BF, device="cuda")
    pool[0, :, :, :C], pool[1, :, :, :C] = x["k"].cuda(), x["v"].cuda()
    arrays = {n: x[n].cuda() for n in ("weights", "positions", "lengths")}
    new_weights, new_positions = torch.empty(B, H, N, device="cuda"), torch.empty(B, H, N, dtype=torch.int32, device="cuda")
    kept, new_lengths = torch.empty(B, H, N, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    pos = torch.tensor([55, 50], dtype=torch.int32, device="cuda")

    def struct(first, slots, weights, positions):
        return _lib.Cache(k=pool[0, :, :, first:].data_ptr(), v=pool[1, :, :, first:].data_ptr(), weights=weights.data_ptr(),
                          positions=positions.data_ptr(), lengths=arrays["lengths"].data_ptr(), dtype=_lib.DF11_BF16, batch=B,
                          kv_heads=H, slots=slots, dim=D, stride_batch=H * (C + N) * D, stride_head=(C + N) * D, stride_slot=D)

    old, new = struct(0, C, arrays["weights"], arrays["positions"]), struct(C, N, new_weights, new_positions)
    _lib.check(_lib.lib().df11_cache_compact(ctypes.byref(old), pos.data_ptr(), N, 4, ctypes.byref(new), kept.data_ptr(),
                                             new_lengths.data_ptr(), torch.cuda.current_stream().cuda_stream), "compact")
    want = ref.cache_compact(x["positions"], x["weights"], x["lengths"], pos.cpu(), N, 4)
    assert torch.equal(kept.cpu(), want)
    at = want.clamp(min=0).long()
    rows = at.unsqueeze(-1).expand(B, H, N, D)
    for i, n in enumerate(("k", "v")):
        assert torch.equal(pool[i, :, :, :C].cpu(), x[n])
        assert torch.equal(pool[i, :, :, C:].cpu(), torch.where((want >= 0).unsqueeze(-1), x[n].gather(2, rows), 0))


@pytest.mark.parametrize("path", ["few shared rows", "many shared rows", "own positions", "cache", "window"])
def test_float16_keeps_small_probabilities(path):
    """Every 32nd key has a logit of 17.046875, the others 0: 2^-24.6 of it each.
    Only they have values (1000): half as much again would come out if their
    probabilities were held as multiples of 2^-24 of the greatest.  The bound:
    the result's rounding, 2^-12 for the sums, and a step of 2^-31 of the
    greatest probability (half of it an error) for each of the 31 others, and
    half of the result's own smallest step."""
    n, big = 512, 17.046875
    k, v = torch.zeros(n, 1, 64, dtype=HF), torch.full((n, 1, 64), 1000.0, dtype=HF)
    k[::32, :, 0], v[::32] = big, 0.0
    batch, tokens, heads = {"few shared rows": (1, 1, 4), "many shared rows": (24, 1, 4), "own positions": (3, 1, 4),
                            "cache": (2, 1, 1), "window": (2, 40, 1)}[path]
    q = torch.zeros(batch, tokens, heads, 64, dtype=HF, device="cuda")
    q[..., 0] = 8.0
    k, v = k.cuda(), v.cuda()
    lengths = torch.full((batch,), n, dtype=torch.int32, device="cuda")
    if "shared" in path:
        out = serve.prefix_attention(q, k, v, k.expand(batch, n, 1, 64), v.expand(batch, n, 1, 64), 0 * lengths, scale=0.125)
    elif path == "own positions":
        out = serve.prefix_attention(q, k[:0], v[:0], k.expand(batch, n, 1, 64), v.expand(batch, n, 1, 64), lengths, scale=0.125)
    else:
        cache = serve.BoundedCache(k.view(1, 1, n, 64).repeat(batch, 1, 1, 1), v.view(1, 1, n, 64).repeat(batch, 1, 1, 1),
                                   torch.zeros(batch, 1, n, device="cuda"),
                                   torch.arange(n, dtype=torch.int32, device="cuda").repeat(batch, 1, 1), lengths)
        out = serve.cache_attention(q, cache, lengths, scale=0.125)
    small = np.exp(-big)
    want = 31 * small * 1000 / (1 + 31 * small)
    bound = (2.0 ** -11 + 2.0 ** -11 + 2.0 ** -12) * want + 2.0 ** -32 * 31 * 1000 + 2.0 ** -25
    off = float((out.double() - want).abs().max())
    assert off <= bound, (off, bound, want)
