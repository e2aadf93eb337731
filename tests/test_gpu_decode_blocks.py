"""The decoding loop (spec_verification_gb300/decode.py) over an 8-bit cache whose blocks have factors of their own:
prompts attended as they come from the projection, steps over the cache."""
import numpy as np
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


def _model(**kw):
    from spec_verification_gb300 import decode
    return decode.Model(**{**dict(vocab=997, layers=2, width=256, q_heads=4, kv_heads=2, head_dim=64, seed=3), **kw})


@pytest.mark.parametrize("drafts,page,block", [(3, 16, 16), (0, 64, 32), (4, 64, 16)])
def test_generated_tokens_are_the_models(drafts, page, block):
    from spec_verification_gb300 import decode
    model = _model()
    rng = np.random.default_rng(5)
    prompts = [rng.integers(0, 20, n).tolist() for n in (2, 17, 40, 64, 1)]
    decoder = decode.Decoder(model, 5, 64 + 12 * (drafts + 1), drafts, page_size=page, cache_dtype="e4m3", block_tokens=block)
    texts, gained = decode.generate(decoder, prompts, 12)
    assert all(g >= 12 for g in gained)
    assert decoder.kv_len.tolist() == [len(t) - 1 for t in texts]
    held = [p for r, n in enumerate(decoder.kv_len.tolist()) for p in decoder.block_table[r, :-(-n // page)].tolist()]
    assert sorted(held + decoder.free_pages[:decoder.free_count.item()].tolist()) == list(range(decoder.plan.num_pages))
    for text, prompt in zip(texts, prompts):
        logits = _plain_logits(model, text)
        for at in range(len(prompt), len(text)):
            row = logits[at - 1]
            assert row[text[at]] >= row.max() - 4.0  # 8-bit values, as in tests/test_gpu_decode.py


@pytest.mark.parametrize("weights", [1.0, 3000.0])
def test_hidden_states_over_the_cache_are_the_models(weights):
    """Prompts, then pieces of texts, against the model without a cache in 32 bits: bounds as in tests/test_gpu_decode_edges.py
    (0.15 with 8-bit values), also where keys and values are far beyond what 8 bits hold without factors."""
    from spec_verification_gb300 import decode, kv
    model = _model(seed=12)
    for layer in model.layers:  # values beyond 448: their factors are what holds them; the projection after takes it back
        layer["qkv"][6 * 64:] *= weights
        layer["out"] /= weights
    decoder = decode.Decoder(model, 3, 100, 4, cache_dtype="e4m3", block_tokens=16)
    g = torch.Generator().manual_seed(3)
    texts = [torch.randint(0, 997, (n,), generator=g).tolist() for n in (3, 50, 81)]
    states = [[] for _ in texts]
    for n, pieces in enumerate(((1, 30, 47), (1, 19, 1), (1, 0, 5), (0, 1, 28))):
        at = [len(s) for s in states]
        hidden, _ = decoder.forward([t[a:a + n] for t, a, n in zip(texts, at, pieces)], whole=n == 0)
        kv.ss_kv_commit(decoder.plan, decoder.block_table, decoder.kv_len, decoder.free_pages, decoder.free_count, decoder.seq_len)
        assert decoder.status.tolist() == [0, 0, 0]
        for s, part in zip(states, hidden.float().split(list(pieces))):
            s.extend(part)
    for r, (text, state) in enumerate(zip(texts, states)):
        want = _plain_logits(model, text)
        got = torch.stack(state) @ model.embed.float().T
        error = (got - want).norm(dim=-1) / want.norm(dim=-1)
        assert len(state) == len(text) and error.max() <= 0.15, error.max().item()
        prompt = (1, 30, 47)[r]
        assert error[:prompt].max() <= 0.05  # 16-bit attention


def test_a_second_batch_of_prompts_reads_the_cache():
    from spec_verification_gb300 import decode
    model = _model()
    rng = np.random.default_rng(9)
    first, second = ([rng.integers(0, 997, n).tolist() for n in (20, 33)] for _ in range(2))
    both = [a[:-1] + b for a, b in zip(first, second)]
    one = decode.Decoder(model, 2, 200, 2, cache_dtype="e4m3", block_tokens=16)
    one.prompt(first)
    one.prompt(second)
    assert one.kv_len.tolist() == [len(b) - 1 for b in both]
    gained = one.step([b[-1] for b in both], [[], []])
    for text, g in zip(both, gained):
        row = _plain_logits(model, text)[-1]
        assert row[g[0]] >= row.max() - 4.0


def test_blocks_that_do_not_fit_are_refused():
    from spec_verification_gb300 import decode
    for kw in (dict(cache_dtype="bf16", block_tokens=16), dict(cache_dtype="e4m3", block_tokens=32), dict(cache_dtype=None, block_tokens=16)):
        with pytest.raises(ValueError):
            decode.Decoder(_model(), 1, 40, 1, **kw)
