"""ss_attend_prompt where a CTA takes many units one after the other, and what rows that are none leave alone: against 64
bits with the bounds of tests/test_gpu_kv_prompt.py, or bit for bit; and infinite keys."""
import math

import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_kv_prompt import U, Prompts, _i32, reference  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _env():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from spec_verification_gb300 import build
    build.build()


def units_to_a_cta(lengths, hq, hkv, dim, spare=3):
    """(units of the call, CTAs, tiles of rows of a unit): the launch of ss_attend_prompt, from its description: a tile of rows has
    whole tokens of as many query heads as fill 115 of 128 rows, of a key head's heads in as few parts as do."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    group, most = hq // hkv, 0
    first = -(-group // 128)
    for parts in range(first, max(8, first) + 1):
        heads = -(-group // parts)
        filled = group * (128 // heads) // parts
        if filled > most:
            most, tokens, chunks, whole = filled, 128 // heads, parts, 32 % heads == 0
        if most >= 115:
            break
    total = sum(lengths) + spare
    few = total * hq <= 256 * sms or total <= (3 * tokens if whole else 200) * len(lengths)
    tiles = 2 if dim == 128 and not few else 1
    ctas = (2 if tiles == 1 and dim <= 128 else 1) * sms
    return sum(-(-n // (tiles * tokens)) for n in lengths) * hkv * chunks, ctas, tiles


# Lengths are such that a prompt's last tile of rows is partly filled, so that rows that leave by way of shared memory and
# rows that leave from registers follow one another in a CTA.
LONG = [1000, 37, 900, 3, 1500, 2100, 450, 333, 129]
SHORT = [1 + 37 * i % 199 for i in range(110)]
HANDED = [
    # lengths, hq, hkv, dim, type, tiles of rows
    (LONG, 16, 8, 256, "bf16", 1),                     # 64 tokens to a tile: whole ones leave by way of the queries' room
    (LONG, 40, 8, 256, "f16", 1),                      # 25 tokens of 5 heads: stores from registers
    ([170] * 40 + [5, 64, 65], 16, 8, 256, "f16", 1),  # short units
    (SHORT, 16, 8, 128, "bf16", 1),
    (SHORT, 40, 8, 128, "f16", 1),
    (LONG + [2600], 32, 8, 128, "bf16", 2),
    (LONG + [2000], 40, 8, 128, "f16", 2),
    (LONG + [1800], 28, 4, 64, "bf16", 1),
    (SHORT, 32, 8, 64, "f16", 1),                      # heads that divide 32
]


@pytest.mark.parametrize("lengths,hq,hkv,dim,kind,tiles", HANDED)
@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 70)])
def test_many_units_to_a_cta(lengths, hq, hkv, dim, kind, tiles, window, sinks):
    """At least five units to a CTA: every barrier between units takes both parities more than once."""
    units, ctas, of = units_to_a_cta(lengths, hq, hkv, dim)
    assert units >= 5 * ctas and of == tiles, (units, ctas, of)
    p = Prompts(lengths, hq, hkv, dim, kind, seed=dim + hq)
    p.run(window, sinks)
    p.check(window, sinks)
    assert p.status.tolist() == [0] * len(lengths)
    first = p.out.clone()
    for _ in range(3):  # whichever CTA takes which unit
        p.out.fill_(7.0)
        p.run(window, sinks)
        torch.cuda.synchronize()
        assert torch.equal(first, p.out)


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


@pytest.mark.parametrize("dim,kind", [(128, "bf16"), (64, "f16"), (256, "bf16")])
def test_infinite_keys_weigh_nothing_or_everything(dim, kind):
    """A first key whose scores are all -inf: as if it were not there, and its own token, which sees nothing else, gives zeros
    and -inf.  Whose scores are +inf: no number for any that sees it."""
    n0, n = 200, 100
    p = Prompts([n0, n], 4, 2, dim, kind)
    q = p.q[n0:n0 + n, 2:]
    q[..., 5] = -q[..., 5].abs() - 0.1
    p.k[n0, 1, 5] = math.inf
    p.run()
    torch.cuda.synchronize()
    got, lse = p.out[n0:n0 + n, 2:].double(), p.lse[n0:n0 + n, 2:].double()
    assert torch.all(got[0] == 0) and torch.all(lse[0] == -math.inf)
    # without the key: token t of the rest sees the keys 1 .. t
    k, v = p.k[n0 + 1:n0 + n, 1:].double(), p.v[n0 + 1:n0 + n, 1:].double()
    want, want_lse, weighted, plain, size = reference(q[1:].double(), k, v, p.scale)
    off = dim * 2.0 ** -23 * size + 2.0 ** -20
    tol = U[kind] * want.abs() * (1 + 2.0 ** -10) + (U[kind] + 2 * off[..., None]) * weighted + 2.0 ** -25
    if kind == "f16":
        tol = tol + 2.0 ** -25 * plain
    assert torch.all((got[1:] - want).abs() <= tol)
    assert torch.all((lse[1:] - want_lse).abs() <= 2 * off + 2.0 ** -22 * want_lse.abs())
    others = p.out[:n0 + n].clone()
    q[..., 5] = -q[..., 5]
    p.run()
    torch.cuda.synchronize()
    bad = ~torch.isfinite(p.out[:n0 + n].double())
    expect = torch.zeros_like(bad)
    expect[n0:, 2:] = True
    assert torch.equal(bad, expect)
    assert torch.equal(others[~expect], p.out[:n0 + n][~expect])
