"""Generation (generate.py) where the sequences' room and the wishes' masks end."""
import pytest

torch = pytest.importorskip("torch")
from huffman_decode_df11_amd import generate, serve  # noqa: E402

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a GPU", allow_module_level=True)

VOCAB = 512


@pytest.fixture(scope="module")
def model():
    return generate.Decoder(generate.Config(vocab=VOCAB), seed=3)


def _generator(model, **more):
    prompt = torch.randint(VOCAB, (40,), generator=torch.Generator().manual_seed(4))
    return generate.Generator(model, prompt, batch=2, budget=24, recent=8, seed=5, **more)


@pytest.mark.parametrize("drafts", [0, 2])
def test_masks_are_not_copied(model, monkeypatch, drafts):
    """One row of bits for all sequences and drafts, read where it lies."""
    seen = []

    class Spy:
        def __getattr__(self, name):
            return getattr(serve, name)

        def adjust_logits(self, logits, *rest, mask, **more):
            seen.append(mask.data_ptr())
            return serve.adjust_logits(logits, *rest, mask=mask, **more)

    monkeypatch.setattr(generate, "serve", Spy())
    g = _generator(model, drafts=drafts, room=30, wishes=generate.Wishes(allowed=torch.arange(VOCAB) % 3 != 1))
    out, _ = g.generate(6)
    assert seen and set(seen) == {g.wishes["mask"].data_ptr()}
    assert all(t % 3 != 1 for s in out for t in s)


@pytest.mark.parametrize("bits", [16, 4])
def test_rounds_end_with_the_room(model, bits):
    """A round that might pass the page table or the history is refused, and leaves everything as it was."""
    g = _generator(model, drafts=2, room=11, cache_bits=bits, wishes=generate.Wishes(presence=0.1))
    rounds = 0
    with pytest.raises(ValueError, match="more room"):
        while rounds < 12:
            g.round()
            rounds += 1
            assert int(g.own_count.max()) <= 11
    assert rounds >= 3
    before = [t.clone() for t in (g.own_count, g.history, g.last)]
    with pytest.raises(ValueError, match="more room"):
        g.round()
    assert all(torch.equal(a, b) for a, b in zip(before, (g.own_count, g.history, g.last)))
