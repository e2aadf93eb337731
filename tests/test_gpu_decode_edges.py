"""The decoding loop (spec_verification_gb300/decode.py) where prompts have nothing to cache."""
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
