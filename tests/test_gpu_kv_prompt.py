"""ss_attend_prompt on the GPU against 64-bit torch.

Bounds, as in tests/test_gpu_kv.py: the output is rounded once (u of its type, 2^-8 or 2^-11); every weight is rounded
to that type for the product with the values (u of it; in f16 also by 2^-25 where it is subnormal, with the largest
weight of the first tile at 2^7 and none smaller than that by more than 2^15 later, so 2^-25 of the largest is plenty)
and comes from a score with D 32-bit roundings of sums of |q k| and a 2^x good to 2^-20.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.fixture(scope="module", autouse=True)
def _env():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from spec_verification_gb300 import build
    build.build()


def _kv():
    from spec_verification_gb300 import kv
    return kv


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def reference(q, k, v, scale, window=0, sinks=0):
    """One prompt: q [n, hq, d], k, v [n, hkv, d] in 64 bits.  Returns out, lse and, for the bounds, sum w |v| / sum w, sum |v| / sum w
    (w = 1 at the largest score) and the largest sum |q k| scale."""
    n, hq, d = q.shape
    g = hq // k.shape[1]
    outs = [[], [], [], [], []]
    t = torch.arange(n, device=q.device)
    see = t[None] <= t[:, None]
    if window:
        see &= (t[None] > t[:, None] - window) | (t[None] < sinks)
    for h in range(hq):
        kk, vv = k[:, h // g], v[:, h // g]
        s = (q[:, h] @ kk.T * scale).masked_fill(~see, -math.inf)
        top = s.amax(1, keepdim=True)
        w = torch.where(see, torch.exp(s - top), 0.0)
        z = w.sum(1, keepdim=True)
        size = (q[:, h].abs() @ kk.abs().T * scale).masked_fill(~see, 0.0).amax(1)
        for x, y in zip(outs, (w @ vv / z, (top + torch.log(z))[:, 0], w @ vv.abs() / z, see.double() @ vv.abs() / z, size)):
            x.append(y)
    return tuple(torch.stack(x, 1) for x in outs)


class Prompts:
    def __init__(self, lengths, hq, hkv, dim, kind, seed=0, size=1.5, spare=3):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.lengths, self.dim, self.kind, self.scale = lengths, dim, kind, dim ** -0.5
        t = self.tokens = sum(lengths)
        heads = hq + 2 * hkv
        # one projection's output, whose rows have a gap; tokens past the last prompt hold NaN
        wide = torch.randn(t + spare, heads * dim + 8, generator=g, device="cuda")
        wide[:, :hq * dim] *= size
        wide[t:] = math.nan
        wide = wide.to(TYPES[kind])
        self.q, self.k, self.v = (wide[:, a * dim:b * dim].view(t + spare, b - a, dim) for a, b in ((0, hq), (hq, hq + hkv), (hq + hkv, heads)))
        self.cu = _i32([0] + np.cumsum(lengths).tolist())
        self.band = torch.full((t + spare, hq * dim + 16), 7.0, device="cuda").to(TYPES[kind])
        self.out = self.band[:, :hq * dim].view(-1, hq, dim)
        self.lse = torch.full((t + spare, hq), 7.0, device="cuda")
        self.status = _i32([0] * len(lengths))
        self.plan = _kv().Plan(max_rows=len(lengths), max_tokens=t + spare, q_heads=hq, kv_heads=hkv, head_dim=dim, page_size=16, num_pages=1,
                               max_blocks=1, dtype=kind)
        self.workspace = torch.zeros(self.plan.workspace_bytes, dtype=torch.uint8, device="cuda")

    def run(self, window=0, sinks=0, **kw):
        args = dict(out=self.out, row_status=self.status, workspace=self.workspace, scale=self.scale, window=window, sinks=sinks, lse=self.lse)
        _kv().ss_attend_prompt(self.plan, self.q, self.k, self.v, self.cu, **{**args, **kw})

    def check(self, window=0, sinks=0, skip=(), lengths=None):
        torch.cuda.synchronize()
        at = 0
        for r, n in enumerate(lengths or self.lengths):
            here = slice(at, at + n)
            at += n
            if n == 0 or r in skip:
                continue
            want, lse, weighted, plain, size = reference(self.q[here].double(), self.k[here].double(), self.v[here].double(), self.scale, window, sinks)
            off = self.dim * 2.0 ** -23 * size + 2.0 ** -20  # of a weight, relative
            tol = U[self.kind] * want.abs() * (1 + 2.0 ** -10) + (U[self.kind] + 2 * off[..., None]) * weighted + 2.0 ** -25
            if self.kind == "f16":
                tol = tol + 2.0 ** -25 * plain
            got = self.out[here].double()
            assert torch.all((got - want).abs() <= tol), (r, ((got - want).abs() / tol).max().item())
            assert torch.all((self.lse[here].double() - lse).abs() <= 2 * off + 2.0 ** -22 * lse.abs())
        assert torch.all(self.out[at:] == 7.0) and torch.all(self.lse[at:] == 7.0)
        assert torch.all(self.band[:, self.out.shape[1] * self.dim:] == 7.0)
        assert int(self.workspace[:4096].view(torch.int32)[:256].abs().sum()) == 0  # counters are left at zero


CASES = [
    # lengths, hq, hkv, dim, type
    ([1], 1, 1, 64, "bf16"),
    ([60], 8, 2, 128, "bf16"),
    ([1, 2, 3, 0, 5, 31, 33], 8, 2, 128, "bf16"),
    ([127, 128, 129], 2, 2, 128, "f16"),
    ([300, 1, 0, 257], 8, 2, 64, "f16"),
    ([700], 7, 1, 128, "bf16"),
    ([0, 0, 130, 0], 71, 1, 64, "bf16"),
    ([10, 40], 130, 1, 64, "f16"),             # more query heads to a key head than a tile has rows
    ([3, 90], 600, 2, 64, "bf16"),
    ([200, 75], 66, 2, 128, "bf16"),           # 33 query heads to a key head
    ([450, 300], 95, 1, 128, "f16"),           # 32, 32 and 31 heads
    ([40, 70], 76, 2, 256, "bf16"),            # 38 heads in five parts, the last of 6
    ([500, 129, 3], 4, 2, 256, "bf16"),
    ([257, 64], 10, 2, 256, "f16"),
    ([1100, 900], 4, 1, 128, "bf16"),
    ([513], 3, 3, 64, "bf16"),
    ([1 + 13 * i % 140 for i in range(200)], 6, 2, 64, "bf16"),
    ([1] * 70, 4, 4, 128, "f16"),
]


@pytest.mark.parametrize("lengths,hq,hkv,dim,kind", CASES)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (50, 3), (128, 0), (200, 1000), (130, 129)])
def test_prompts(lengths, hq, hkv, dim, kind, window, sinks):
    p = Prompts(lengths, hq, hkv, dim, kind, seed=len(lengths) + dim)
    p.run(window, sinks)
    p.check(window, sinks)
    assert p.status.tolist() == [0] * len(lengths)
    first = p.out.clone()
    p.run(window, sinks)
    torch.cuda.synchronize()
    assert torch.equal(first, p.out)


# prompts long enough for two tiles of query rows to a unit (more than 200 tokens a prompt, tokens * q_heads above 256 an SM)
LONG = [
    ([3000, 1, 500, 0, 1700], 8, 2, "bf16"),   # 32 tokens to a tile of rows: whole ones leave by way of shared memory
    ([2900, 40], 14, 2, "f16"),                # 18 tokens, 126 rows: stores from registers
    ([2560, 130], 16, 16, "bf16"),             # 128 tokens: the first tile of rows has fewer key tiles
    ([700] * 8, 8, 1, "f16"),
    ([600, 610], 64, 1, "bf16"),               # two tokens
]


@pytest.mark.parametrize("lengths,hq,hkv,kind", LONG)
@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 0), (700, 70)])
def test_two_tiles_of_rows(lengths, hq, hkv, kind, window, sinks):
    p = Prompts(lengths, hq, hkv, 128, kind, seed=hq)
    p.run(window, sinks)
    p.check(window, sinks)
    assert p.status.tolist() == [0] * len(lengths)
    first = p.out.clone()
    p.run(window, sinks, lse=None)
    torch.cuda.synchronize()
    assert torch.equal(first, p.out)


@pytest.mark.parametrize("kind,hq", [("bf16", 8), ("f16", 14)])
def test_two_tiles_of_rows_with_values_that_are_not_finite(kind, hq):
    p = Prompts([3000, 1700], hq, 2, 128, kind)
    p.v[1010, 1, 7], p.v[2999, 0, 3] = math.inf, math.nan
    p.run(window=300)
    torch.cuda.synchronize()
    got, half = p.out[:4700].double(), hq // 2
    expect = torch.zeros_like(got, dtype=torch.bool)
    expect[1010:1310, half:, 7] = True
    expect[2999, :half, 3] = True
    assert torch.equal(~torch.isfinite(got), expect)
    p.v[1010, 1, 7] = p.v[2999, 0, 3] = 0.0
    p.run(window=300)
    torch.cuda.synchronize()
    clean = p.out[:4700].double()
    assert torch.all(((got - clean).abs() <= 2 * U[kind] * clean.abs() + 2.0 ** -16)[~expect])


def test_two_tiles_of_rows_in_a_graph_and_on_odd_outputs():
    p = Prompts([3000, 2200], 8, 2, 128, "bf16")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run()
    for lengths in ([5200, 0], [1, 5199], [2600, 2600]):
        p.out.fill_(7.0)
        p.lse.fill_(7.0)
        p.cu.copy_(_i32([0] + np.cumsum(lengths).tolist()))
        graph.replay()
        p.check(lengths=lengths)
    wide = torch.full((5203, 8 * 128 + 8), 7.0, device="cuda").to(torch.bfloat16)
    out = wide[:, 8:].view(5203, 8, 128)
    p.run(out=out)
    torch.cuda.synchronize()
    assert torch.equal(out[:5200], p.out[:5200]) and torch.all(out[5200:] == 7.0) and torch.all(wide[:, :8] == 7.0)


def test_long_prompt():
    """Many units to a CTA; the last rows of a long prompt, and its first, against 64 bits."""
    p = Prompts([5000, 3], 8, 1, 128, "bf16")
    p.run()
    p.check()


@pytest.mark.parametrize("kind,dim", [("bf16", 128), ("f16", 64), ("bf16", 256)])
def test_sharp_scores(kind, dim):
    """Scores of thousands: the running maximum moves, weights underflow."""
    p = Prompts([400, 60], 4, 2, dim, kind, size=400.0)
    p.run()
    p.check()


@pytest.mark.parametrize("kind,dim", [("bf16", 128), ("f16", 256)])
def test_scores_beyond_32_bit_steps(kind, dim):
    p = Prompts([200], 4, 2, dim, kind)
    p.scale = 2.0 ** 24
    p.run()
    torch.cuda.synchronize()
    got, lse = p.out[:200].double(), p.lse[:200].double()
    assert torch.all(torch.isfinite(got)) and torch.all(torch.isfinite(lse))
    _, want, _, _, size = reference(p.q[:200].double(), p.k[:200].double(), p.v[:200].double(), p.scale)
    assert torch.all((lse - want).abs() <= dim * 2.0 ** -22 * size)
    assert torch.all(got.abs().amax(-1) > 0)


@pytest.mark.parametrize("kind,dim,hq", [("bf16", 128, 8), ("f16", 64, 6), ("bf16", 256, 4), ("f16", 128, 2)])
@pytest.mark.parametrize("wild", [math.inf, -math.inf, math.nan])
def test_values_that_are_not_finite_stay_with_who_sees_them(kind, dim, hq, wild):
    """In values of a token that later ones see, in one past their window, and in keys that nobody sees."""
    lengths = [300, 290]
    p = Prompts(lengths, hq, 2, dim, kind)
    p.v[150, 1, 7] = wild                        # prompt 0: tokens 150 .. 229 with the window of 80
    p.v[299, 0, 3] = wild                        # its last token: seen by itself, next to prompt 1's first
    p.run(window=80)
    torch.cuda.synchronize()
    got, half = p.out[:590].double(), hq // 2
    expect = torch.zeros_like(got, dtype=torch.bool)
    expect[150:230, half:, 7] = True
    expect[299, :half, 3] = True
    assert torch.equal(~torch.isfinite(got), expect)
    p.v[150, 1, 7] = p.v[299, 0, 3] = 0.0
    p.run(window=80)
    torch.cuda.synchronize()
    clean = p.out[:590].double()
    # a tile that is added key by key differs in the order of its sums: a rounding of the output and of 2^-20 of its terms
    assert torch.all(((got - clean).abs() <= 2 * U[kind] * clean.abs() + 2.0 ** -16)[~expect])


def test_keys_that_are_not_finite_stay_with_who_sees_them():
    p = Prompts([200, 100], 4, 2, 128, "bf16")
    p.k[120, 0, 5] = math.nan
    p.k[200, 1, 5] = math.inf                    # the first of prompt 1: everyone in it sees it
    p.run()
    torch.cuda.synchronize()
    bad = ~torch.isfinite(p.out[:300].double()).all(-1)
    expect = torch.zeros(300, 4, dtype=torch.bool, device="cuda")
    expect[120:200, :2] = True
    assert torch.equal(bad[:200], expect[:200]) and not bad[200:, :2].any()


def test_many_prompts():
    """8192 prompts, most of them of one token or none, and bad ones among them."""
    lengths = [(0, 1, 2, 1, 5, 1, 40, 1)[i % 8] for i in range(8192)]
    p = Prompts(lengths, 4, 2, 64, "bf16", spare=5)
    cu = p.cu.clone()
    p.cu[4000], p.cu[8192] = -1, p.tokens + 6    # prompts 3999 and 4000, and the last one
    p.run()
    torch.cuda.synchronize()
    bad = [r for r, s in enumerate(p.status.tolist()) if s]
    assert bad == [3999, 4000, 8191] and set(p.status.tolist()) == {0, 1 << 9}
    at = cu.tolist()
    for r in list(range(40)) + list(range(3990, 4010)) + list(range(8150, 8192)):
        here = slice(at[r], at[r + 1])
        if r in bad:
            assert torch.all(p.out[here] == 7.0)
        elif lengths[r]:
            want, _, weighted, _, size = reference(p.q[here].double(), p.k[here].double(), p.v[here].double(), p.scale)
            tol = U["bf16"] * want.abs() * (1 + 2.0 ** -10) + (U["bf16"] + 2 * (64 * 2.0 ** -23 * size + 2.0 ** -20)[..., None]) * weighted + 2.0 ** -25
            assert torch.all((p.out[here].double() - want).abs() <= tol), r
    # all others: as if computed with good prefix sums
    first = p.out.clone()
    p.cu = cu
    p.run()
    torch.cuda.synchronize()
    good = torch.ones(p.out.shape[0], dtype=torch.bool, device="cuda")
    for r in bad:
        good[at[r]:at[r + 1]] = False
    assert torch.equal(first[good], p.out[good])


@pytest.mark.parametrize("dim,hq", [(64, 6), (128, 4), (256, 2)])
def test_outputs_on_16_byte_boundaries(dim, hq):
    """Rows that are not 32-byte aligned are written in halves."""
    p = Prompts([150, 33], hq, 2, dim, "bf16")
    wide = torch.full((186, hq * dim + 8), 7.0, device="cuda").to(torch.bfloat16)
    out = wide[:, 8:].view(186, hq, dim)
    p.run()
    p.run(out=out)
    torch.cuda.synchronize()
    assert torch.equal(out[:183], p.out[:183]) and torch.all(out[183:] == 7.0) and torch.all(wide[:, :8] == 7.0)


def test_bad_prefix_sums_are_reported():
    p = Prompts([30, 50, 20, 40], 4, 2, 64, "bf16")
    p.cu = _i32([0, 30, 80, 70, 140])            # the third decreases; the fourth is tokens 70 .. 139
    p.run()
    torch.cuda.synchronize()
    assert p.status.tolist() == [0, 0, 1 << 9, 0]
    p.status.zero_()
    p.out.fill_(7.0)
    p.cu = _i32([-5, 30, 80, 100, 2 ** 31 - 1])
    p.run()
    torch.cuda.synchronize()
    assert p.status.tolist() == [1 << 9, 0, 0, 1 << 9]
    assert torch.all(p.out[:30] == 7.0) and torch.all(p.out[100:] == 7.0) and torch.all(p.out[30:100] != 7.0)


def test_on_another_stream_and_in_a_graph():
    p = Prompts([200, 40, 77], 8, 2, 128, "bf16")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    p.run(stream=side)
    side.synchronize()
    p.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p.run()
    for lengths in ([1, 1, 1], [0, 317, 0], [100, 100, 117]):
        p.out.fill_(7.0)
        p.lse.fill_(7.0)
        p.cu.copy_(_i32([0] + np.cumsum(lengths).tolist()))
        graph.replay()
        p.check(lengths=lengths)


def test_the_cached_attention_agrees():
    """Prompts over their own keys and values, and the same by way of a 16-bit cache."""
    kv = _kv()
    lengths, hq, hkv, dim, page = [100, 37], 8, 2, 128, 16
    p = Prompts(lengths, hq, hkv, dim, "bf16", spare=0)
    p.run()
    plan = kv.Plan(max_rows=2, max_tokens=137, max_new=100, q_heads=hq, kv_heads=hkv, head_dim=dim, page_size=page, num_pages=12, max_blocks=8)
    cache = torch.zeros(2, 12, page, hkv, dim, dtype=torch.bfloat16, device="cuda")
    table = torch.arange(16, dtype=torch.int32, device="cuda").view(2, 8).clamp(max=11)
    for r, (a, n) in enumerate(((0, 100), (100, 37))):
        for c, x in zip(cache, (p.k, p.v)):
            t = torch.arange(n, device="cuda")
            c[table[r, t // page].long(), t % page] = x[a:a + n]
    out, status = torch.empty(137, hq, dim, dtype=torch.bfloat16, device="cuda"), _i32([0, 0])
    kv.ss_attend(plan, p.q, cache[0], cache[1], table, _i32(lengths), p.cu, out=out, row_status=status, scale=p.scale,
                 workspace=torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert torch.all((out.double() - p.out[:137].double()).abs() <= 4 * U["bf16"] * (1 + out.double().abs()))


def test_wrong_arguments_are_refused():
    from spec_verification_gb300 import native
    p = Prompts([20, 3], 4, 2, 64, "bf16", spare=0)

    def refused(code, call=None, **change):
        args = dict(q=p.q, k=p.k, v=p.v, cu_seq=p.cu, out=p.out, row_status=p.status, workspace=p.workspace, scale=p.scale)
        with pytest.raises(native.SSError) as e:
            _kv().ss_attend_prompt(p.plan, **{**args, **change})
        assert e.value.code == code, (change.keys(), str(e.value))

    refused(-1, q=p.q[:, :3])
    refused(-1, k=p.k[:-1])
    refused(-1, v=p.v.half())
    refused(-1, out=p.out[:-1])
    refused(-1, k=p.k.cpu())
    refused(-1, cu_seq=p.cu.long())
    refused(-1, B=3)
    refused(-1, B=0)
    refused(-1, scale=0.0)
    refused(-1, scale=math.inf)
    refused(-1, scale=math.nan)
    refused(-1, window=-1)
    refused(-1, sinks=-1)
    refused(-1, lse=torch.zeros(5, 4, device="cuda"))
    refused(-4, workspace=p.workspace[:256])
    refused(-2, workspace=torch.zeros(p.plan.workspace_bytes + 64, dtype=torch.uint8, device="cuda")[64:])
    odd = torch.zeros(23, 4 * 64 + 4, dtype=torch.bfloat16, device="cuda")[:, :256].view(23, 4, 64)
    refused(-2, q=odd)
    refused(-2, out=odd)
    raw = torch.zeros(23 * 128 + 8, dtype=torch.bfloat16, device="cuda")[4:23 * 128 + 4].view(23, 2, 64)
    refused(-2, k=raw)
    none = torch.zeros(0, 4, 64, dtype=torch.bfloat16, device="cuda")
    _kv().ss_attend_prompt(p.plan, none, none[:, :2], none[:, :2], p.cu, out=none, row_status=p.status, workspace=p.workspace, scale=1.0)
    torch.cuda.synchronize()
    assert p.status.tolist() == [0, 0]
