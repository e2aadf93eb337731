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
