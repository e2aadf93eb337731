"""The decoding loop (spec_verification_gb300/decode.py) where prompts do not fit, or have nothing to cache."""
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_decode import _plain_logits  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _env():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from spec_verification_gb300 import build
    build.build()


def _decoder(rows, most, **kw):
    from spec_verification_gb300 import decode
    model = decode.Model(vocab=997, layers=1, width=128, q_heads=2, kv_heads=1, head_dim=64, seed=8)
    return decode.Decoder(model, rows, most, 2, **kw)


@pytest.mark.parametrize("prompts,pages,bit", [
    ([[1] * 40, [2] * 40], 4, 1 << 11),     # three pages each, four in all
    ([[1] * 20, [2] * 60], None, 1 << 12),  # four pages, three to a table row
])
def test_a_prompt_that_does_not_fit_is_reported(prompts, pages, bit):
    decoder = _decoder(2, 40, num_pages=pages)
    with pytest.raises(RuntimeError) as e:
        decoder.prompt(prompts)
    assert f"['0x0', '{hex(bit)}']" in str(e.value)
    # nothing is kept, and the same decoder still takes prompts that fit
    assert decoder.kv_len.tolist() == [0, 0] and decoder.free_count.item() == decoder.plan.num_pages
    decoder.prompt([p[:18] for p in prompts])
    assert decoder.kv_len.tolist() == [17, 17]
    assert all(decoder.step([1, 2], [[], []]))


def test_prompts_of_one_token_have_nothing_to_cache():
    from spec_verification_gb300 import decode
    decoder = _decoder(3, 100)
    texts, gained = decode.generate(decoder, [[5], [6], [7]], 4)
    assert all(g >= 4 for g in gained)
    assert decoder.kv_len.tolist() == [len(t) - 1 for t in texts]
    for text in texts:
        logits = _plain_logits(decoder.model, text)
        for at in range(1, len(text)):
            assert logits[at - 1][text[at]] >= logits[at - 1].max() - 1.5  # as in tests/test_gpu_decode.py


@pytest.mark.parametrize("cache,most", [("bf16", 0.05), ("e4m3", 0.15)])
def test_hidden_states_over_the_cache_are_the_models(cache, most):
    """Texts taken in pieces, against the model without a cache in 32 bits.  Some 26 roundings to bf16 lie between input and
    logits (2^-8 / sqrt(3) each, in the mean: 0.012 of the norm together); 8-bit keys and values add 2^-4 / sqrt(3) to those
    of an attention.  Up to four times that."""
    from spec_verification_gb300 import decode, kv
    model = decode.Model(vocab=997, layers=2, width=256, q_heads=4, kv_heads=2, head_dim=64, seed=12)
    decoder = decode.Decoder(model, 3, 100, 4, cache_dtype=cache)
    g = torch.Generator().manual_seed(3)
    texts = [torch.randint(0, 997, (n,), generator=g).tolist() for n in (3, 50, 81)]
    states = [[] for _ in texts]
    for pieces in ((1, 30, 47), (1, 19, 1), (1, 0, 5), (0, 1, 28)):
        at = [len(s) for s in states]
        hidden, _ = decoder.forward([t[a:a + n] for t, a, n in zip(texts, at, pieces)])
        kv.ss_kv_commit(decoder.plan, decoder.block_table, decoder.kv_len, decoder.free_pages, decoder.free_count, decoder.seq_len)
        assert decoder.status.tolist() == [0, 0, 0]
        for s, part in zip(states, hidden.float().split(list(pieces))):
            s.extend(part)
    for text, state in zip(texts, states):
        want = _plain_logits(model, text)
        got = torch.stack(state) @ model.embed.float().T
        error = (got - want).norm(dim=-1) / want.norm(dim=-1)
        assert len(state) == len(text) and error.max() <= most, error.max().item()
