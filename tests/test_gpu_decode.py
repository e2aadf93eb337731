"""The decoding loop (spec_verification_gb300/decode.py): every token that it
generates is the argmax of the same model computed without a cache, in 32 bits,
up to the rounding of 16-bit activations; pages and lengths add up."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import kv_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _env():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from spec_verification_gb300 import build
    build.build()


def _plain_logits(model, text):
    """The model over a whole text without a cache, in 32 bits."""
    x = model.embed[torch.tensor(text, device=model.device)].float()
    n, hq, hkv, d = len(text), model.q_heads, model.kv_heads, model.head_dim
    positions = torch.arange(n, device=model.device)
    for layer in model.layers:
        w = {k: v.float() for k, v in layer.items()}
        qkv = model.norm(x) @ w["qkv"].T
        q, k, v = (p.view(n, -1, d) for p in qkv.split([hq * d, hkv * d, hkv * d], 1))
        q = ref.rope(q, w["q_norm"], positions, model.inv_freq, False)
        k = ref.rope(k, w["k_norm"], positions, model.inv_freq, False)
        out = ref.attend(q, k, v.double(), 0, d ** -0.5)[0].float()
        x = x + out.reshape(n, hq * d) @ w["out"].T
        x = model.feed_forward(w, x)
    return model.norm(x) @ model.embed.float().T


@pytest.mark.parametrize("cache,drafts", [("bf16", 4), ("bf16", 0), ("e4m3", 3)])
def test_generated_tokens_are_the_models(cache, drafts):
    from spec_verification_gb300 import decode
    model = decode.Model(vocab=997, layers=2, width=256, q_heads=4, kv_heads=2, head_dim=64, seed=3)
    rng = np.random.default_rng(5)
    prompts = [rng.integers(0, 20, n).tolist() for n in (2, 17, 40, 64)]
    decoder = decode.Decoder(model, 4, 64 + 12 * (drafts + 1), drafts, cache_dtype=cache)
    texts, gained = decode.generate(decoder, prompts, 12)
    assert all(g >= 12 for g in gained)
    assert decoder.kv_len.tolist() == [len(t) - 1 for t in texts]
    held = [p for r, n in enumerate(decoder.kv_len.tolist()) for p in decoder.block_table[r, :-(-n // 16)].tolist()]
    free = decoder.free_pages[:decoder.free_count.item()].tolist()
    assert sorted(held + free) == list(range(decoder.plan.num_pages))
    # 16-bit activations through two layers move a logit of these (spread about 16) by some tenths; 8-bit values more
    slack = 4.0 if cache == "e4m3" else 1.5
    for text, prompt in zip(texts, prompts):
        logits = _plain_logits(model, text)
        for at in range(len(prompt), len(text)):
            row = logits[at - 1]
            assert row[text[at]] >= row.max() - slack, (at, row[text[at]].item(), row.max().item())


def test_rejected_drafts_leave_no_trace():
    """Wrong drafts in every step, as many as fit: the same texts as without drafts, up to near ties."""
    from spec_verification_gb300 import decode
    model = decode.Model(vocab=997, layers=2, width=256, q_heads=4, kv_heads=2, head_dim=64, seed=4)
    rng = np.random.default_rng(6)
    prompts = [rng.integers(0, 20, n).tolist() for n in (3, 30, 33)]
    plain, _ = decode.generate(decode.Decoder(model, 3, 200, 0), prompts, 10)
    noise = np.random.default_rng(7)
    wrong = lambda text, most: noise.integers(0, 997, most).tolist()  # noqa: E731
    drafted, gained = decode.generate(decode.Decoder(model, 3, 200, 5), prompts, 10, draft=wrong)
    same = [sum(a == b for a, b in zip(p[len(q):], d[len(q):])) for p, d, q in zip(plain, drafted, prompts)]
    assert sum(same) >= 0.8 * sum(min(10, g) for g in gained), same


def test_sampled_decoding_runs_and_finished_rows_return_their_pages():
    from spec_verification_gb300 import decode
    model = decode.Model(vocab=997, layers=1, width=128, q_heads=2, kv_heads=1, head_dim=64, seed=8)
    decoder = decode.Decoder(model, 3, 100, 2, greedy=False)
    prompts = [[1, 2, 3], [4, 5] * 10, [7] * 33]
    decoder.prompt(prompts)
    decoder.step([p[-1] for p in prompts], [[9], [], [7, 7]])
    decoder.step([1, 2, 3], [[], [5], []], finished=[0, 1, 0])
    assert decoder.kv_len.tolist()[1] == 0
    used = sum(-(-n // 16) for n in decoder.kv_len.tolist())
    assert decoder.free_count.item() == decoder.plan.num_pages - used
