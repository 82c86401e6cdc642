"""Speculative generation over the operators together (generate.py): greedy
tokens against the same model in float64 with a full cache, and the bounded
caches' state behind refused drafts."""
import pytest

torch = pytest.importorskip("torch")
from huffman_decode_df11_amd import generate, serve  # noqa: E402

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)


def _reference_logits(model, ids):
    """Logits of every position of one sequence, in float64 on the CPU."""
    c = model.config
    w = lambda lin: lin.decoded_weight().double().cpu()   # noqa: E731

    def norm(x):
        return x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6)

    def turn(x):
        angle = torch.arange(x.shape[0], dtype=torch.float64)[:, None, None] * model.inverse.double().cpu()
        a, b = x.chunk(2, -1)
        return torch.cat([a * angle.cos() - b * angle.sin(), b * angle.cos() + a * angle.sin()], -1)

    x = model.embed(ids.cuda()).double().cpu()
    n = ids.numel()
    mask = torch.ones(n, n, dtype=torch.bool).tril()
    for layer in model.layers:
        h = norm(x)
        q = turn((h @ w(layer.q).T).view(n, c.heads, c.dim))
        k = turn((h @ w(layer.k).T).view(n, c.kv_heads, c.dim)).repeat_interleave(c.heads // c.kv_heads, 1)
        v = (h @ w(layer.v).T).view(n, c.kv_heads, c.dim).repeat_interleave(c.heads // c.kv_heads, 1)
        s = torch.einsum("qhd,khd->hqk", q, k) * c.dim ** -0.5
        p = torch.softmax(torch.where(mask, s, -torch.inf), -1)
        x = x + torch.einsum("hqk,khd->qhd", p, v).reshape(n, -1) @ w(layer.o).T
        h = norm(x)
        x = x + (torch.nn.functional.silu(h @ w(layer.gate).T) * (h @ w(layer.up).T)) @ w(layer.down).T
    return norm(x) @ w(model.head).T


def test_greedy_tokens_are_the_full_models():
    """Each emitted token is the reference's likeliest, or short of it by no
    more than bfloat16 rounding makes of a logit near 4 (activations and
    probabilities rounded to 2^-8, some 20 roundings: 4 * 2^-8 * 20 = 0.32)."""
    model = generate.Decoder(generate.Config(vocab=1024), seed=3)
    prompt = torch.randint(1024, (300,), generator=torch.Generator().manual_seed(4))
    g = generate.Generator(model, prompt, batch=3, budget=64, recent=16, drafts=3, room=64, temperature=0.0, seed=5)
    out, taken = g.generate(20)
    assert 0.0 <= taken <= 3.0
    assert out[0] == out[1] == out[2] and len(out[0]) == 20
    ids = torch.cat([prompt, torch.tensor(out[0])])
    logits = _reference_logits(model, ids[:-1])[299:]
    short = logits.max(1).values - logits.gather(1, torch.tensor(out[0])[:, None])[:, 0]
    assert float(short.max()) < 0.32, short


def test_sampling_fills_and_evicts():
    """Sampled sequences differ; the bounded caches stay full, hold each
    position once and the latest ones whole."""
    model = generate.Decoder(generate.Config(vocab=1024), seed=6)
    prompt = torch.randint(1024, (100,), generator=torch.Generator().manual_seed(7))
    g = generate.Generator(model, prompt, batch=4, budget=48, recent=12, drafts=2, room=80, temperature=1.0, seed=8)
    out, _ = g.generate(30)
    assert len({tuple(s) for s in out}) == 4
    nxt = g._positions().cpu()
    for cache in g.caches:
        assert cache.lengths.tolist() == [48] * 4
        for b in range(4):
            for h in range(model.config.kv_heads):
                live = [p for p in cache.positions[b, h].tolist() if p < int(nxt[b]) and p != serve.NO_TOKEN]
                assert len(live) == len(set(live))
                # all but the newest token (its key comes with the next round) of the latest positions
                assert set(range(int(nxt[b]) - 9, int(nxt[b]))) <= set(live)


def test_command():
    import sys
    argv, sys.argv = sys.argv, ["generate", "--batch", "2", "--prompt", "70", "--new", "9", "--budget", "32"]
    try:
        generate.main()
    finally:
        sys.argv = argv


@pytest.mark.parametrize("prompt,budget,drafts,seed", [(100, 48, 4, 8), (100, 48, 4, 9), (40, 200, 4, 10), (100, 64, 3, 11)])
def test_refused_drafts_leave_the_bounded_caches(prompt, budget, drafts, seed, monkeypatch):
    """After every round, full caches and not full ones: no position twice and
    none from behind the tokens that stay.  About half of the drafts are
    refused (the drafter's probabilities are doubled before the verification)."""
    verify = serve.verify_drafts
    monkeypatch.setattr(generate.serve, "verify_drafts", lambda d, p, u, q: verify(d, p, u, 2.0 * q))
    model = generate.Decoder(generate.Config(vocab=1024), seed=6)
    ids = torch.randint(1024, (prompt,), generator=torch.Generator().manual_seed(7))
    g = generate.Generator(model, ids, batch=4, budget=budget, recent=12, drafts=drafts, room=120, temperature=1.0, seed=seed)
    refused = 0
    for _ in range(12):
        _, taken = g.round()
        refused += int((drafts - taken).sum())
        nxt = g._positions().cpu()
        for cache in g.caches:
            for b in range(4):
                for h in range(model.config.kv_heads):
                    there = cache.positions[b, h, :int(cache.lengths[b])].tolist()
                    there = [p for p in there if p != serve.NO_TOKEN]
                    assert len(there) == len(set(there)) and max(there) < int(nxt[b])
    assert refused > 40


def test_prompt_of_one_token():
    """Nothing before the sequences' own positions: greedy tokens are the full model's (the bound above)."""
    model = generate.Decoder(generate.Config(vocab=1024), seed=3)
    prompt = torch.tensor([17])
    out, _ = generate.Generator(model, prompt, batch=2, budget=24, recent=8, drafts=3, room=64, temperature=0.0).generate(30)
    assert out[0] == out[1] and len(out[0]) == 30
    logits = _reference_logits(model, torch.cat([prompt, torch.tensor(out[0])])[:-1])
    short = logits.max(1).values - logits.gather(1, torch.tensor(out[0])[:, None])[:, 0]
    assert float(short.max()) < 0.32, short
    with pytest.raises(ValueError, match="prompt"):
        generate.Generator(model, prompt[:0], batch=2)


def test_without_drafts():
    """One token a round, the full model's (the bound above)."""
    model = generate.Decoder(generate.Config(vocab=1024), seed=3)
    prompt = torch.randint(1024, (70,), generator=torch.Generator().manual_seed(4))
    out, taken = generate.Generator(model, prompt, batch=2, budget=24, recent=8, drafts=0, room=20, temperature=0.0).generate(12)
    assert taken == 0.0 and out[0] == out[1] and len(out[0]) == 12
    logits = _reference_logits(model, torch.cat([prompt, torch.tensor(out[0])])[:-1])[69:]
    short = logits.max(1).values - logits.gather(1, torch.tensor(out[0])[:, None])[:, 0]
    assert float(short.max()) < 0.32, short
