"""ss_attend_prompt: what rows that are none leave alone, bit for bit."""
import math

import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_kv_prompt import Prompts, _i32  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _env():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from spec_verification_gb300 import build
    build.build()


NEIGHBOURS = [
    # lengths, hq, hkv, dim, type
    ([197, 61], 8, 2, 128, "bf16"),
    ([197, 61], 8, 2, 128, "f16"),
    ([3005, 61], 16, 4, 128, "bf16"),  # two tiles of rows
    ([131, 61], 28, 4, 64, "bf16"),
    ([131, 61], 4, 2, 256, "bf16"),
    ([1, 61], 8, 2, 256, "f16"),
]


@pytest.mark.parametrize("lengths,hq,hkv,dim,kind", NEIGHBOURS)
@pytest.mark.parametrize("wild", ["large", math.inf, -math.inf, math.nan])
def test_a_prompt_does_not_depend_on_its_neighbour(lengths, hq, hkv, dim, kind, wild):
    """The next prompt's queries, and what lies past the last one's, share tiles of rows with a prompt's last tokens: whatever they
    are, its bits stay."""
    n = lengths[0]
    for used in (lengths, lengths[:1]):
        p = Prompts(lengths, hq, hkv, dim, kind)
        if len(used) == 1:
            p.cu, p.status = _i32([0, n]), _i32([0])
        p.run()
        torch.cuda.synchronize()
        out, lse = p.out[:n].clone(), p.lse[:n].clone()
        p.q[n:] = 0.0
        p.q[n:, :, 3] = (6e4 if kind == "f16" else 2.0 ** 60) if wild == "large" else wild
        p.run()
        torch.cuda.synchronize()
        assert torch.equal(out, p.out[:n]) and torch.equal(lse, p.lse[:n])
        assert p.status.tolist() == [0] * len(used)


@pytest.mark.parametrize("hq,dim,kind", [(76, 256, "bf16"), (76, 64, "f16"), (76, 128, "bf16")])
def test_a_key_heads_queries_do_not_depend_on_the_next_ones(hq, dim, kind):
    """38 query heads to a key head in parts, the last of which is smaller: its tile holds heads of the next key head too."""
    p = Prompts([40, 70], hq, 2, dim, kind)
    p.run()
    torch.cuda.synchronize()
    out, lse = p.out[:110, :38].clone(), p.lse[:110, :38].clone()
    p.q[:, 38:] = 0.0
    p.q[:, 38:, 3] = math.inf
    p.run()
    torch.cuda.synchronize()
    assert torch.equal(out, p.out[:110, :38]) and torch.equal(lse, p.lse[:110, :38])
