"""The quantised cache's operators where values, tiles and layouts meet their
ends: values that a row must not see beside ones that it does, groups near the ends of
a type's range, and outputs that lie on inputs."""
import pytest

torch = pytest.importorskip("torch")

import quantized_reference as ref  # noqa: E402
from huffman_decode_df11_amd import _lib, serve  # noqa: E402

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

BF, HF, I32 = torch.bfloat16, torch.float16, torch.int32
INF, NAN = float("inf"), float("nan")
MANY = 112   # rows that share a key head's keys up to which values are not made


def _gen(seed):
    return torch.Generator().manual_seed(seed)


def _randn(g, *shape, dtype=BF, scale=1.0):
    return (scale * torch.randn(shape, generator=g)).to(dtype)


def _held(k, v):
    """Codes and pairs of rows k, v [pages, H, page, D], on the CPU."""
    (kc, ks, km), (vc, vs, vm) = ref.quantise(k), ref.quantise(v)
    return [ref.packed(kc), ref.packed(vc), torch.stack([ks, km], -1), torch.stack([vs, vm], -1)]


def _on_gpu(parts):
    return serve.QuantizedCache(*(t.cuda() for t in parts))


def _check(q, parts, lengths, table, what, scale=None):
    """Output and lse of every row within their bounds."""
    print("case", what, flush=True)
    n = torch.tensor(lengths, dtype=I32)
    many = q.shape[1] * q.shape[2] // parts[0].shape[1] > MANY
    out, lse = serve.quantized_attention(q.cuda(), _on_gpu(parts), n.cuda(), block_table=table.cuda(), scale=scale, return_lse=True)
    torch.cuda.synchronize()
    want, want_lse, bound = ref.attention(q, parts, n, table, scale, many)
    got, got_lse = out.cpu().double(), lse.cpu().double()
    assert torch.equal(torch.isfinite(got), torch.isfinite(want)), what
    # a result below the type's normal range (2^-14 in float16) is rounded to a whole smallest number, off by up to half of one
    off = (got - want).abs() - bound - torch.finfo(q.dtype).smallest_normal * torch.finfo(q.dtype).eps / 2
    assert float(off.nan_to_num(nan=-1.0).max()) <= 1e-30, (what, float(off.nan_to_num(nan=-1.0).max()))
    return got, got_lse, want_lse


@pytest.mark.parametrize("times", [8.0, 2.0 ** 15, "alone"])
@pytest.mark.parametrize("dtype,D", [(BF, 64), (HF, 64), (BF, 128), (HF, 128), (BF, 256), (HF, 256)])
def test_values_behind_a_tiles_last_key(dtype, D, times):
    """640 rows of 160 tokens are several tiles, whose last keys lie inside a
    step; V of the positions right behind each tile's last one is up to 2^15
    times the others', or the others are zero.  No row of the tile sees them."""
    g = _gen(D)
    T, n, page = 160, 197, 16
    v = _randn(g, 15, 1, page, D, dtype=dtype, scale=2.0 ** -6)
    parts = _held(_randn(g, 15, 1, page, D, dtype=dtype), v)
    table = torch.randperm(15, generator=g)[:13].view(1, 13).to(I32)
    if times == "alone":
        kept, parts[3] = parts[3], torch.zeros_like(parts[3])
    for tile in range(32 if D == 256 else 64, T, 32 if D == 256 else 64):
        for s in (n - T + tile, n - T + tile + 5):   # the first key that the rows before token `tile` do not see
            at = (table[0, s // page].long(), slice(None), s % page)
            parts[3][at] = kept[at] if times == "alone" else parts[3][at] * times
    _check(_randn(g, 1, T, 4, D, dtype=dtype), parts, [n], table, (dtype, D, times))


def _write(k):
    """Codes and pairs of rows k [n, 64] as they are written, and the same rows' in 64 bits."""
    n = k.shape[0]
    per = -(-n // 16)
    cache = serve.QuantizedCache.empty(per, 1, 16, 64, dtype=k.dtype)
    rows, table = k[None, :, None].cuda(), torch.arange(per, dtype=I32, device="cuda").view(1, per)
    serve.quantized_write(cache, rows, rows, torch.zeros(1, dtype=I32, device="cuda"), block_table=table)
    codes, step, least = ref.quantise(k)
    for c, s in ((cache.k_codes, cache.k_scales), (cache.v_codes, cache.v_scales)):
        assert torch.equal(s.cpu().flatten(0, 2)[:n], torch.stack([step, least], -1))
        yield ref.unpacked(c.cpu().flatten(0, 2)[:n]), codes


@pytest.mark.parametrize("dtype", [BF, HF])
def test_codes_of_values_on_a_border_over_a_tiny_least_value(dtype):
    """A border of the steps from 0 is missed by as much as the least value
    lies above 0 (or passed, below 0), however little that is."""
    g, rows = _gen(1), []
    groups = [(2.0 ** -24, 2.0, 60.0), (2.0 ** -24, 7.5, 15.0), (2.0 ** -20, 0.5, 15.0)]
    if dtype == BF:
        groups += [(2.0 ** -30, 1.0, 30.0), (2.0 ** -26, 3.0, 30.0), (2.0 ** -30, 0.5, 15.0), (2.0 ** -50, 10.5, 15.0)]
    for least, on, greatest in groups:
        row = torch.full((64,), on, dtype=torch.float64)
        row[::8], row[3::8], row[4::8], row[7::8] = least, least, greatest, greatest
        rows.append(row)
    for _ in range(3000):   # values on borders of steps that are powers of two, over least values down to 2^-40 of one
        step = 2.0 ** int(torch.randint(-6, 7, (1,), generator=g))
        row = (torch.randint(0, 15, (64,), generator=g).double() + 0.5) * step
        least = step * 2.0 ** -float(torch.randint(0, 41, (1,), generator=g)) * (1 if len(rows) % 2 else -1)
        row[:2], row[2:4] = least, 15 * step
        rows.append(row)
    for got, want in _write(torch.stack(rows).to(dtype)):
        wrong = (got != want).any(-1).nonzero().flatten()
        assert not wrong.numel(), (wrong.numel(), wrong[:5].tolist(), [rows[i][:4].tolist() for i in wrong[:2]])


@pytest.mark.parametrize("T", [1, 10, 65])
@pytest.mark.parametrize("dtype", [BF, HF])
def test_keys_at_the_ends_of_the_range(dtype, T):
    """Groups that reach the type's greatest number: the step is rounded, so
    that the greatest code may stand for more than that."""
    g = _gen(T)
    top = float(torch.finfo(dtype).max)
    least = -top if dtype == HF else -2.0 ** 120
    k = _randn(g, 6, 1, 16, 128, dtype=dtype)
    k[:, :, ::3, 5], k[:, :, ::3, 9], k[:, :, 1::3, 4], k[:, :, 1::3, 7] = top, least, -top, top
    parts = _held(k, _randn(g, 6, 1, 16, 128, dtype=dtype))
    past = (15 * parts[2][..., 0].double() + parts[2][..., 1].double()).max()
    assert past > top
    # logits of a size near 1 at the least and greatest numbers
    small = 2.0 ** -12 if dtype == HF else 2.0 ** -112
    q, scale = _randn(g, 1, T, 2, 128, dtype=dtype, scale=small), 2.0 ** -4 if dtype == HF else 2.0 ** -16
    _, lse, want_lse = _check(q, parts, [70], torch.tensor([[3, 1, 0, 5, 2]], dtype=I32), (dtype, T), scale)
    # logits: sums of |q| (143 or 31) step in float32, K to 2^-16 (bfloat16) or 2^-20 of its values
    reach = scale * float(q.double().abs().sum(-1).max()) * float(parts[2][..., 0].double().abs().max())
    assert float((lse - want_lse).abs().max()) <= 2.0 ** -12 + (2.0 ** -20 * 143 + 2.0 ** -16 * 15) * reach


@pytest.mark.parametrize("n", [70, 3000])
@pytest.mark.parametrize("scale", [2.0 ** 120, 2.0 ** 126.9])
def test_many_rows_over_values_at_the_end_of_the_range(scale, n):
    """V of bfloat16 up to its greatest number, in one range of keys and in several."""
    g = _gen(n)
    per = -(-n // 16)
    v = (torch.randn((per, 1, 16, 64), generator=g).clamp(-1.0, 1.0).double() * scale).to(BF)
    parts = _held(_randn(g, per, 1, 16, 64), v)
    assert torch.isfinite(v).all() and torch.isfinite(parts[3]).all()
    _check(_randn(g, 1, 65, 2, 64), parts, [n], torch.randperm(per, generator=g).view(1, per).to(I32), (scale, n))


def test_many_rows_over_float16_values_from_end_to_end():
    """One position's V spans float16's range and its greatest code stands for
    65536; the others' are 2^20 smaller and less."""
    g = _gen(7)
    v = _randn(g, 6, 1, 16, 128, dtype=HF, scale=2.0 ** -9)
    v[4, 0, 3, ::2], v[4, 0, 3, 1::2] = 65504.0, -65504.0
    v[4, 0, 3, 4:8] = torch.tensor([-65504.0, 65504.0, -65504.0, 65504.0])
    parts = _held(_randn(g, 6, 1, 16, 128, dtype=HF), v)
    assert float((15 * parts[3][..., 0].double() + parts[3][..., 1].double()).max()) == 65536.0
    got, _, _ = _check(_randn(g, 1, 65, 2, 128, dtype=HF), parts, [90], torch.tensor([[3, 4, 0, 5, 2, 1]], dtype=I32), "end to end")
    assert torch.isfinite(got).all()


@pytest.mark.parametrize("dtype", [BF, HF])
def test_finite_rows_are_read_back_finite(dtype):
    """A code may stand for more than the type's greatest number (the step is
    rounded): it is read as that; what has no number stays without one."""
    top = float(torch.finfo(dtype).max)
    rows = torch.zeros((5, 64), dtype=dtype)
    rows[0, ::2], rows[0, 1::2] = (torch.linspace(0, 1, 32) * top).to(dtype), (torch.linspace(-1, 1, 32) * top).to(dtype)
    rows[1, 2:4], rows[1, 8:10] = top, -top if dtype == HF else -2.0 ** 120
    rows[2, 7], rows[3, 6], rows[4, 5] = NAN, INF, -INF
    cache = serve.QuantizedCache.empty(1, 1, 16, 64, dtype=dtype)
    one = lambda x: torch.full((1,), x, dtype=I32, device="cuda")   # noqa: E731
    serve.quantized_write(cache, rows[None, :, None].cuda(), rows[None, :, None].flip(1).cuda(), one(0))
    cache.k_scales[0, 0, 6, 0, 1] = INF   # as no write makes them
    cache.k_scales[0, 0, 7, 1, 0] = -INF
    k, v = (x.cpu()[0, :, 0] for x in serve.quantized_read(cache, one(9), 9))
    codes, step, least = ref.quantise(rows)
    want = codes.double() * ref.spread(step.double(), 64) + ref.spread(least.double(), 64)
    assert want[:2].max() > top
    want = want.clamp(-top, top).float().to(dtype)
    for got, w in ((k[:5], want), (v[:5], want.flip(0))):
        assert torch.equal(torch.isnan(got), torch.isnan(w)) and torch.equal(got.nan_to_num(), w.nan_to_num())
    assert torch.isfinite(k[:2]).all() and float(k[:2].max()) == top
    assert not torch.isfinite(k[6, ::2]).any() and not k[6, 1::2].any() and not torch.isfinite(k[7, 1::2]).any()


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("T", [1, 20, 65, 200])
def test_lse_of_large_logits(T, dtype):
    """Logits of hundreds (bfloat16: thousands) against their own bound, which
    keys held in one number of the type would leave."""
    g = _gen(T)
    parts = _held(_randn(g, 14, 1, 16, 128, dtype=dtype), _randn(g, 14, 1, 16, 128, dtype=dtype))
    q = _randn(g, 1, T, 2, 128, dtype=dtype, scale=100.0 if dtype == HF else 1000.0)
    n, scale = 201, 128 ** -0.5
    table = torch.randperm(14, generator=g).view(1, 14).to(I32)
    _, lse, want = _check(q, parts, [n], table, (T, dtype))
    at = table[0].long()
    k = ref.values(parts[0][at, 0], parts[2][at, 0]).flatten(0, 1)[:n]
    step = ref.spread(parts[2][at, 0][..., 0].double(), 128).flatten(0, 1)[:n]
    size = q[0].double().abs()
    # A logit is a float32 sum of terms up to a step times the offset and 15, taken off again, and of values: 16 roundings
    # of the whole each.  Many rows: K's values in two numbers of the type, made in float32 from 16 + a code.
    u = ref.UNIT[dtype]
    logit = 2.0 ** -20 * (step * (ref.OFF[dtype] + 15.0) + k.abs())
    if 2 * T > MANY:
        logit = logit + u * u * k.abs() + 2.0 ** -19 * step
    # the greatest of the row's logits' errors; the exponentials' and sums'; m and the logarithm beside it in float32
    bound = scale * (size @ logit.t()).amax(-1) + 2.0 ** -16 + 2.0 ** -22 * want[0].abs()
    assert bool(((lse - want)[0].abs() <= bound).all()), float(((lse - want)[0].abs() / bound).max())
    once = k.to(dtype).double()
    seen = torch.arange(n) < n - T + 1 + torch.arange(T).view(T, 1, 1)
    rough = torch.logsumexp((scale * q[0].double() @ once.t()).masked_fill(~seen, -INF), -1)
    if 2 * T > MANY:
        assert float(((rough - want[0]).abs() > bound).double().mean()) > 0.5


@pytest.mark.parametrize("n", [70, 3000])
@pytest.mark.parametrize("seen", ["by all", "by some", "by the last"])
def test_many_rows_over_bfloat16_values_from_end_to_end(seen, n):
    """One position's V reaches bfloat16's greatest number, and its greatest
    code stands for more; the others' are of a size near 1 and come out as such where it is not seen."""
    g = _gen(n)
    per, T = -(-n // 16), 65
    at = dict(zip(("by all", "by some", "by the last"), (n - T - 3, n - 30, n - 1)))[seen]
    v = _randn(g, per, 1, 16, 64)
    top = float(torch.finfo(BF).max)
    table = torch.randperm(per, generator=g).view(1, per).to(I32)
    page = int(table[0, at // 16])
    v[page, 0, at % 16, :2], v[page, 0, at % 16, 2:4] = top, -2.0 ** 120
    parts = _held(_randn(g, per, 1, 16, 64), v)
    assert float((15 * parts[3][..., 0].double() + parts[3][..., 1].double()).max()) > top
    got, _, _ = _check(_randn(g, 1, T, 2, 64), parts, [n], table, (seen, n))
    before = got[0, :max(0, at - (n - T))]
    assert not before.numel() or float(before.abs().max()) < 8.0


@pytest.mark.parametrize("bad", [NAN, INF])
@pytest.mark.parametrize("dtype,D", [(BF, 64), (HF, 128), (BF, 256)])
def test_no_numbers_behind_a_tiles_last_key(dtype, D, bad):
    """The first position that a tile's last row does not see has no number for
    V (or no value but 0): the rows before it are the same to the bit, of several tiles and ranges."""
    g = _gen(D)
    T, page = 160, 16
    tokens = 32 if D == 256 else 64
    for n in (197, 1500):
        per = -(-n // page)
        parts = _held(_randn(g, per, 1, page, D, dtype=dtype), _randn(g, per, 1, page, D, dtype=dtype))
        table = torch.randperm(per, generator=g).view(1, per).to(I32)
        q, lengths = _randn(g, 1, T, 4, D, dtype=dtype).cuda(), torch.tensor([n], dtype=I32).cuda()
        for first in (tokens, 2 * tokens, T - 1):
            s = n - T + first
            outs = []
            for x in (0.0, bad):
                changed = [p.clone() for p in parts]
                changed[3][table[0, s // page].long(), :, s % page] = x
                outs.append(serve.quantized_attention(q, _on_gpu(changed), lengths, block_table=table.cuda()))
            assert torch.equal(outs[0][:, :first], outs[1][:, :first]) and torch.isfinite(outs[0]).all(), (n, first)
            assert not torch.isfinite(outs[1][:, first:]).any(), (n, first)
