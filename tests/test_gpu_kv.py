"""The KV-cache operators on the GPU against plain forms (tests/kv_reference.py).

Bounds.  u(t) = finfo(t).eps / 2 is the most that one rounding to type t moves
a value, relative to it.  Rotary store: the arithmetic is a norm (sum of D
squares, square root, two products), a rotation (two products, a sum) and, for
8 bits, a quotient, in 32 bits: 16 roundings of 2^-24 at the size of the pair,
then one rounding to the output type; cos and sin of 32 bits add 2^-22.
Attention: the output is rounded once (u of its type); every softmax weight
is rounded to the product's type (u of it; f16 weights also by 2^-25 where they
are subnormal) and comes from a score with D 32-bit roundings of sums of |q k|
and a 2^x good to 2^-20.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import kv_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11, "e4m3": 2.0 ** -4}


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


# ------------------------------------------------------------------ pages
def _pool(kv_len, page, blocks, spare, seed):
    rng = np.random.default_rng(seed)
    used = [-(-max(0, n) // page) for n in kv_len]
    pages = sum(used) + spare
    ids = rng.permutation(pages).tolist()
    table, at = [], 0
    for u in used:
        table.append(ids[at:at + u] + [-1] * (blocks - u))
        at += u
    free = ids[at:] + [-7] * at  # entries past the count are stale
    return table, free, spare, pages


def _plan(rows, tokens, page, pages, blocks, **kw):
    kw = {"q_heads": 4, "kv_heads": 2, "head_dim": 64, **kw}
    return _kv().Plan(max_rows=rows, max_tokens=max(1, tokens), page_size=page, num_pages=max(1, pages), max_blocks=blocks, **kw)


PAGES = [
    # kv_len, new, page, blocks, spare
    ([0], [1], 16, 4, 4),
    ([0], [0], 16, 1, 1),
    ([16, 15, 17, 0, 31], [1, 1, 1, 16, 17], 16, 8, 40),
    ([5, 40, 16], [3, 100, 0], 32, 16, 9),
    ([1, 1, 1, 1], [20, 1, 20, 20], 16, 4, 2),        # the pool runs out; a row that needs no page is still served
    ([60, 3, 64], [5, 70, 1], 16, 4, 50),             # rows past their table
    ([100, 7], [0, 0], 16, 8, 3),
    ([3, 2], [2000, 700], 16, 200, 400),              # pieces of prompts
]


@pytest.mark.parametrize("kv_len,new,page,blocks,spare", PAGES)
def test_append(kv_len, new, page, blocks, spare):
    _check_append(kv_len, new, page, blocks, spare)


@pytest.mark.parametrize("rows,most,longest,page", [(300, 9, 700, 16), (1025, 1, 50, 32), (37, 200, 3000, 64), (8192, 2, 40, 16)])
def test_append_many_rows(rows, most, longest, page):
    rng = np.random.default_rng(rows)
    kv_len, new = rng.integers(0, longest, rows).tolist(), rng.integers(0, most + 1, rows).tolist()
    _check_append(kv_len, new, page, -(-(longest + most) // page), rows // 2 * (1 + most // page))


def _check_append(kv_len, new, page, blocks, spare, table=None):
    kv = _kv()
    made, free, count, pages = _pool(kv_len, page, blocks, spare, 3)
    table = table or made
    cu = [0] + np.cumsum(new).tolist()
    want = ref.append(table, kv_len, free, count, cu, page, blocks, pages, max(1, cu[-1]))
    plan = _plan(len(new), cu[-1], page, pages, blocks)
    t, l, f, c = _i32(table), _i32(kv_len), _i32(free), _i32([count])
    slots, positions = _i32([99] * (cu[-1] + 3)), _i32([99] * (cu[-1] + 3))
    seq, status = _i32([99] * len(new)), _i32([99] * len(new))
    for _ in range(2):  # an append can be repeated
        kv.ss_kv_append(plan, t, l, f, c, _i32(cu), slots=slots, positions=positions, seq_len=seq, row_status=status)
    torch.cuda.synchronize()
    assert t.tolist() == want[0]
    assert slots.tolist() == want[1] + [99] * 3
    assert positions.tolist() == want[2] + [99] * 3
    assert seq.tolist() == want[3]
    assert status.tolist() == want[4]
    assert l.tolist() == kv_len and f.tolist() == free and c.tolist() == [count]
    return want


def test_append_reports_bad_pages_and_parameters():
    table, free, count, pages = _pool([20, 20, 20], 16, 4, 3, 5)
    table[1][1] = pages          # past the cache
    table[2][1] = -5
    got = _check_append([20, 20, 20], [1, 1, 1], 16, 4, 3, table)
    assert got[4] == [0, 1 << 13, 1 << 13]
    got = _check_append([20, -3, 20], [2, 2, 2], 16, 4, 3)
    assert got[4] == [0, 1 << 4, 0]


@pytest.mark.parametrize("kv_len,new,page,blocks,spare", PAGES)
@pytest.mark.parametrize("how", ["all", "counts", "finished"])
def test_commit(kv_len, new, page, blocks, spare, how):
    rng = np.random.default_rng(11)
    counts = None if how == "all" else [int(rng.integers(-1, n + 2)) for n in new]
    finished = [int(rng.integers(0, 2)) for _ in new] if how == "finished" else None
    _check_commit(kv_len, new, page, blocks, spare, counts, 0 if how == "all" else 1, finished)


@pytest.mark.parametrize("rows,most,longest,page", [(300, 9, 700, 16), (1025, 1, 50, 32), (37, 200, 3000, 64), (8192, 2, 40, 16)])
def test_commit_many_rows(rows, most, longest, page):
    rng = np.random.default_rng(rows)
    kv_len, new = rng.integers(0, longest, rows).tolist(), rng.integers(0, most + 1, rows).tolist()
    counts, finished = rng.integers(0, most + 1, rows).tolist(), (rng.random(rows) < 0.1).astype(int).tolist()
    _check_commit(kv_len, new, page, -(-(longest + most) // page), rows * (1 + most // page), counts, 1, finished)


def _check_commit(kv_len, new, page, blocks, spare, counts, plus, finished):
    kv = _kv()
    table, free, count, pages = _pool(kv_len, page, blocks, spare, 4)
    cu = [0] + np.cumsum(new).tolist()
    table, _, _, seq, _ = ref.append(table, kv_len, free, count, cu, page, blocks, pages, max(1, cu[-1]))
    want = ref.commit(table, kv_len, free, count, seq, page, counts, plus, finished)
    plan = _plan(len(new), cu[-1], page, pages, blocks)
    t, l, f, c = _i32(table), _i32(kv_len), _i32(free), _i32([count])
    kv.ss_kv_commit(plan, t, l, f, c, _i32(seq), counts=None if counts is None else _i32(counts), plus=plus,
                    finished=None if finished is None else _i32(finished))
    torch.cuda.synchronize()
    assert l.tolist() == want[0]
    assert c.tolist() == [want[2]]
    assert f.tolist() == want[1]
    assert t.tolist() == table
    # every page is in one place: in a row's held blocks or among the free ones
    held = [p for r, n in enumerate(want[0]) for p in table[r][:-(-n // page)]]
    assert sorted(held + f.tolist()[:want[2]]) == list(range(pages))


# ------------------------------------------------------------------ rotary store
def _cache(kind, layout, pages, page, heads, dim, fill):
    shape = (pages, heads, page, dim) if layout == "hnd" else (pages, page, heads, dim)
    t = torch.full(shape, fill, dtype=torch.float32, device="cuda").to(TYPES[kind])
    return t.transpose(1, 2) if layout == "hnd" else t


ROPE = [
    # tokens, hq, hkv, dim, rot, interleaved, norm, type, cache, layout, page
    (1, 1, 1, 64, 64, False, True, "bf16", "bf16", "hnd", 16),
    (7, 8, 2, 128, 128, False, True, "bf16", "bf16", "nhd", 16),
    (33, 5, 5, 128, 48, False, False, "f16", "f16", "hnd", 32),
    (33, 14, 2, 64, 32, True, True, "f16", "f16", "nhd", 64),
    (19, 4, 1, 256, 256, True, False, "bf16", "bf16", "hnd", 128),
    (19, 3, 1, 256, 64, False, True, "f16", "f16", "nhd", 1024),
    (50, 8, 8, 128, 128, False, True, "bf16", "e4m3", "hnd", 16),
    (50, 6, 2, 64, 64, True, False, "f16", "e4m3", "nhd", 16),
    (12, 2, 2, 128, 0, False, True, "bf16", "bf16", "hnd", 16),
    (2600, 6, 2, 64, 64, False, True, "bf16", "bf16", "hnd", 16),   # many tokens: several to a CTA, a ragged end
    (2501, 2, 1, 128, 96, True, True, "f16", "e4m3", "nhd", 32),
]


@pytest.mark.parametrize("tokens,hq,hkv,dim,rot,inter,norm,kind,cache,layout,page", ROPE)
def test_rope_store(tokens, hq, hkv, dim, rot, inter, norm, kind, cache, layout, page):
    kv = _kv()
    g = torch.Generator(device="cuda").manual_seed(tokens + dim)
    pages = -(-tokens // page) + 2
    qkv = (torch.randn(tokens, (hq + 2 * hkv) * dim + 8, generator=g, device="cuda") * 2).to(TYPES[kind])  # rows with a gap
    q, k, v = (x.view(tokens, -1, dim) for x in torch.split(qkv[:, :-8], [hq * dim, hkv * dim, hkv * dim], 1))
    qw, kw = ((1 + 0.3 * torch.randn(2, dim, generator=g, device="cuda")).to(TYPES[kind]) if norm else (None, None))
    positions = torch.randint(0, 2 ** 31 - 1, (tokens,), generator=g, device="cuda").to(torch.int32)
    positions[: tokens // 2] %= 5000
    positions[0] = 0
    slots = torch.randperm(pages * page, generator=g, device="cuda")[:tokens].to(torch.int32)
    if tokens > 5:
        slots[3], slots[5] = -1, pages * page  # stored nowhere
    inv = torch.tensor(kv.rope_frequencies(rot, 10000.0), device="cuda") if rot else None
    low = cache == "e4m3"
    ks, vs = ((0.02 + torch.rand(2, hkv, generator=g, device="cuda") * 0.1) if low else (None, None))
    kc, vc = _cache(cache, layout, pages, page, hkv, dim, 3.0), _cache(cache, layout, pages, page, hkv, dim, 5.0)
    out = torch.full((tokens, hq, dim), 7.0, device="cuda").to(TYPES[kind])
    plan = _plan(1, tokens, page, pages, 1, q_heads=hq, kv_heads=hkv, head_dim=dim, dtype=kind, cache_dtype=cache)
    kv.ss_rope_store(plan, q, k, v, kc, vc, inv, positions, slots, q_out=out, q_weight=qw, k_weight=kw, interleaved=inter,
                     rope_scale=1.25, k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()

    def size(x):  # of a pair, at every value of it: what roundings before the last one are relative to
        y = x.abs()
        if rot:
            a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
            s = y[..., a] + y[..., b]
            y[..., a], y[..., b] = s, s
        return y

    arith = 16 * 2.0 ** -24 + 2.0 ** -22
    # the fixed-point angle against the 64-bit product: positions up to 2^31 leave 2^-20 there
    far = 2.0 ** 31 * 2.0 ** -52
    want = ref.rope(q, qw, positions, inv, inter, scale=1.25)
    assert torch.all((out.double() - want).abs() <= U[kind] * want.abs() + (arith + far) * size(want) * 1.5 + 2.0 ** -25)
    wk = ref.rope(k, kw, positions, inv, inter, scale=1.25)
    wv = v.double()
    filled_k, filled_v = torch.full(kc.shape, 3.0, dtype=torch.float64, device="cuda"), torch.full(kc.shape, 5.0, dtype=torch.float64, device="cuda")
    tol_k, tol_v = torch.zeros_like(filled_k), torch.zeros_like(filled_v)
    good = (slots >= 0) & (slots < pages * page)
    page_of, place = slots[good].long() // page, slots[good].long() % page
    least = 0.0
    if low:
        wk, wv = wk / ks.double()[:, None], wv / vs.double()[:, None]
        least = 2.0 ** -10  # half a step of the smallest 8-bit values
    slack_k = (arith + far) * size(wk) * 1.5 + 2.0 ** -25
    if low:
        wk, wv = wk.clamp(-448, 448), wv.clamp(-448, 448)
    filled_k[page_of, place], filled_v[page_of, place] = wk[good], wv[good]
    tol_k[page_of, place] = (U[cache] * wk.abs() + slack_k * (1 + U[cache]) + least)[good]
    if low:
        tol_v[page_of, place] = (U[cache] * wv.abs() * (1 + 2.0 ** -20) + least)[good]
    assert torch.all((kc.double() - filled_k).abs() <= tol_k)
    assert torch.all((vc.double() - filled_v).abs() <= tol_v)


def test_rope_in_place_and_special_values():
    """q_out may be q; infinities and NaN stay in their own pair and leave unrotated values of their head alone."""
    kv = _kv()
    plan = _plan(1, 8, 16, 4, 1, q_heads=2, kv_heads=1, head_dim=64)
    q = torch.randn(8, 2, 64, device="cuda").bfloat16()
    q[3, 1, 2], q[4, 0, 50] = math.inf, math.nan
    k, v = torch.randn(8, 1, 64, device="cuda").bfloat16(), torch.randn(8, 1, 64, device="cuda").bfloat16()
    kc, vc = _cache("bf16", "hnd", 4, 16, 1, 64, 0.0), _cache("bf16", "hnd", 4, 16, 1, 64, 0.0)
    inv = torch.tensor(kv.rope_frequencies(32), device="cuda")
    positions, slots = torch.arange(8, device="cuda", dtype=torch.int32) + 1, torch.arange(8, device="cuda", dtype=torch.int32)
    apart = torch.empty_like(q)
    kv.ss_rope_store(plan, q, k, v, kc, vc, inv, positions, slots, q_out=apart)
    before = q.clone()
    kv.ss_rope_store(plan, q, k, v, kc, vc, inv, positions, slots, q_out=q)
    torch.cuda.synchronize()
    assert torch.equal(q.view(torch.int16), apart.view(torch.int16))
    wild = ~torch.isfinite(q.float())
    expect = torch.zeros_like(wild)
    expect[3, 1, [2, 18]] = True
    expect[4, 0, 50] = True
    assert torch.equal(wild, expect)
    assert torch.equal(q[..., 32:][~wild[..., 32:]], before[..., 32:][~wild[..., 32:]])


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("scaled", [False, True])
@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_rope_store_8_bits_of_special_values(kind, scaled, dim):
    """Infinities and values beyond the range are held as 448 with their sign, NaN as NaN; nothing is rotated here."""
    kv = _kv()
    plan = _plan(1, 8, 16, 4, 1, q_heads=2, kv_heads=2, head_dim=dim, dtype=kind, cache_dtype="e4m3")
    wild = torch.tensor([math.inf, -math.inf, math.nan, 60000.0, -60000.0, 0.0, 449.0, 2.0], device="cuda").repeat(dim // 8).to(TYPES[kind])
    q, k, v = (torch.zeros(8, 2, dim, device="cuda", dtype=TYPES[kind]) for _ in range(3))
    k[3, 1], v[5, 0] = wild, wild
    factors = torch.tensor([0.5, 0.25], device="cuda") if scaled else None
    kc, vc = _cache("e4m3", "hnd", 4, 16, 2, dim, 0.0), _cache("e4m3", "hnd", 4, 16, 2, dim, 0.0)
    places = torch.arange(8, device="cuda", dtype=torch.int32)
    kv.ss_rope_store(plan, q, k, v, kc, vc, None, places, places, q_out=q, k_scale=factors, v_scale=factors)
    torch.cuda.synchronize()
    for cache, token, head in ((kc, 3, 1), (vc, 5, 0)):
        got = cache.float()
        two = 2.0 / (factors[head].item() if scaled else 1.0)
        want = torch.tensor([448.0, -448.0, math.nan, 448.0, -448.0, 0.0, 448.0, two], device="cuda").repeat(dim // 8)
        assert torch.equal(torch.nan_to_num(got[0, token, head], nan=-1.0), torch.nan_to_num(want, nan=-1.0))
        got[0, token, head] = 0.0
        assert torch.all(got == 0.0)


# ------------------------------------------------------------------ attention
def _held(x, kind, scale):
    """Values as the cache holds them, and in 64 bits."""
    if kind == "e4m3":
        y = (x / scale[None, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn)
        return y, y.double() * scale.double()[None, :, None]
    y = x.to(TYPES[kind])
    return y, y.double()


class Batch:
    """Rows with their own keys and values, scattered over the pages of a cache that holds NaN everywhere else."""

    def __init__(self, new, length, hq, hkv, dim, kind, cache, layout, page, seed=0, spread=1.0):
        kv = _kv()
        g = torch.Generator(device="cuda").manual_seed(seed)
        rows = len(new)
        blocks = max(1, max(-(-n // page) for n in length))
        used = [-(-n // page) for n in length]
        pages = sum(used) + 3
        ids = torch.randperm(pages, generator=g, device="cuda").tolist()
        self.scale, self.hkv, self.kind, self.cache, self.dim, self.page = dim ** -0.5, hkv, kind, cache, dim, page
        low = cache == "e4m3"
        self.ks = 0.01 + 0.05 * torch.rand(hkv, generator=g, device="cuda") if low else None
        self.vs = 0.01 + 0.05 * torch.rand(hkv, generator=g, device="cuda") if low else None
        self.kc, self.vc = (_cache(cache, layout, pages, page, hkv, dim, math.nan) for _ in range(2))
        table = torch.full((rows, blocks), -1, dtype=torch.int32)
        self.k, self.v, at = [], [], 0
        for r, n in enumerate(length):
            k, k64 = _held(torch.randn(n, hkv, dim, generator=g, device="cuda") * spread, cache, self.ks)
            v, v64 = _held(torch.randn(n, hkv, dim, generator=g, device="cuda"), cache, self.vs)
            self.k.append(k64)
            self.v.append(v64)
            mine = ids[at:at + used[r]]
            at += used[r]
            table[r, :used[r]] = torch.tensor(mine, dtype=torch.int32)
            for b, p in enumerate(mine):
                part = slice(b * page, min(n, (b + 1) * page))
                m = part.stop - part.start
                for c, x in ((self.kc, k), (self.vc, v)):
                    if low:
                        c.view(torch.uint8)[p, :m] = x[part].view(torch.uint8)
                    else:
                        c[p, :m] = x[part]
        self.table, self.new, self.length, self.pages = table.cuda(), new, length, pages
        tokens = sum(new)
        wide = (torch.randn(max(1, tokens), hq * dim + 16, generator=g, device="cuda") * 1.5).to(TYPES[kind])
        self.tokens = tokens
        self.q = wide[:, :hq * dim].view(-1, hq, dim)  # rows with a gap
        self.cu = _i32([0] + np.cumsum(new).tolist())
        self.out = torch.full((tokens + 1, hq, dim), 7.0, device="cuda").to(TYPES[kind])
        self.lse = torch.full((tokens + 1, hq), 7.0, device="cuda")
        self.status = _i32([0] * rows)
        self.plan = kv.Plan(max_rows=rows, max_tokens=max(1, tokens), max_new=max(1, max(new)), q_heads=hq, kv_heads=hkv, head_dim=dim,
                            page_size=page, num_pages=pages, max_blocks=blocks, dtype=kind, cache_dtype=cache)
        self.workspace = torch.zeros(self.plan.workspace_bytes, dtype=torch.uint8, device="cuda")

    def run(self, window=0, sinks=0, stream=None):
        _kv().ss_attend(self.plan, self.q, self.kc, self.vc, self.table, _i32(self.length), self.cu, out=self.out,
                        row_status=self.status, workspace=self.workspace, scale=self.scale, window=window, sinks=sinks, lse=self.lse,
                        k_scale=self.ks, v_scale=self.vs, stream=stream)

    def check(self, window=0, sinks=0, hidden=None):
        torch.cuda.synchronize()
        n = self.tokens
        assert torch.all(self.out[n:] == 7.0) and torch.all(self.lse[n:] == 7.0)
        at = 0
        product = "f16" if self.cache == "e4m3" else self.kind
        for r, m in enumerate(self.new):
            want, lse, weighted, plain, size = ref.attend(self.q[at:at + m].double(), self.k[r], self.v[r], self.length[r] - m, self.scale,
                                                          window, sinks, None if hidden is None else hidden.get(r))
            got, got_lse = self.out[at:at + m].double(), self.lse[at:at + m].double()
            at += m
            off = (self.dim * 2.0 ** -23 * size + 2.0 ** -20)  # of a weight, relative
            tol = U[self.kind] * want.abs() * (1 + 2.0 ** -10) + (U[product] + 2 * off[..., None]) * weighted + 2.0 ** -25
            if product == "f16":
                tol = tol + 2.0 ** -25 * plain
            live = torch.isfinite(lse)
            assert torch.all(((got - want).abs() <= tol) | (got == want)), (r, (got - want).abs().max().item())
            assert torch.equal(live, torch.isfinite(got_lse))
            assert torch.all((got_lse - lse)[live].abs() <= (2 * off + 2.0 ** -22 * lse.abs())[live])
            assert torch.all(got_lse[~live] == -math.inf) and torch.all(got[~live] == 0)
        # counters are left at zero
        assert int(self.workspace[:4096].view(torch.int32)[:256].abs().sum()) == 0


ATTEND = [
    # new, length, hq, hkv, dim, type, cache, layout, page
    ([1], [1], 1, 1, 64, "bf16", "bf16", "hnd", 16),
    ([1, 1, 1], [5, 64, 65], 8, 2, 128, "bf16", "bf16", "hnd", 16),
    ([1, 1], [700, 3000], 32, 8, 128, "bf16", "bf16", "nhd", 16),
    ([3, 1, 0, 7], [3, 190, 40, 333], 8, 1, 128, "f16", "f16", "hnd", 32),
    ([5, 2], [129, 1000], 10, 2, 64, "bf16", "bf16", "nhd", 64),
    ([4, 3], [128, 77], 14, 2, 256, "f16", "f16", "hnd", 16),
    ([8, 8, 1], [400, 8, 1], 16, 2, 128, "bf16", "bf16", "hnd", 128),
    ([6, 2], [200, 515], 12, 2, 256, "bf16", "bf16", "nhd", 256),
    ([1, 2, 1], [20, 300, 64], 8, 4, 128, "bf16", "e4m3", "hnd", 16),
    ([9, 1], [300, 1500], 8, 1, 128, "f16", "e4m3", "nhd", 64),
    ([1, 3], [130, 64], 6, 2, 64, "bf16", "e4m3", "hnd", 16),
    ([5, 8], [261, 80], 8, 2, 256, "bf16", "e4m3", "nhd", 16),
    ([100, 40, 1], [100, 333, 50], 4, 2, 128, "bf16", "bf16", "hnd", 16),     # pieces of prompts: several row tiles
    ([70], [200], 3, 1, 64, "f16", "f16", "hnd", 512),
    ([2], [6000], 71, 1, 64, "bf16", "bf16", "nhd", 1024),
    ([1] * 200, [1 + 7 * i % 150 for i in range(200)], 4, 2, 64, "f16", "f16", "hnd", 16),
    ([0, 0, 1], [10, 0, 3], 2, 2, 64, "bf16", "bf16", "hnd", 16),
    ([0, 0], [10, 0], 2, 2, 64, "bf16", "bf16", "hnd", 16),
]


@pytest.mark.parametrize("new,length,hq,hkv,dim,kind,cache,layout,page", ATTEND)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (50, 0), (50, 3), (64, 70), (200, 1000)])
def test_attend(new, length, hq, hkv, dim, kind, cache, layout, page, window, sinks):
    b = Batch(new, length, hq, hkv, dim, kind, cache, layout, page, seed=len(new) + dim)
    b.run(window, sinks)
    b.check(window, sinks)
    assert b.status.tolist() == [0] * len(new)
    first = b.out.clone()
    b.run(window, sinks)  # the same bits again: the join's order is fixed
    torch.cuda.synchronize()
    assert torch.equal(first.view(torch.int16), b.out.view(torch.int16))


ATTEND_8BIT = [
    # the 8-bit kernels by query rows and columns: one buffer of 128 query rows, copies of 64, all columns at once
    ([9, 4], [700, 130], 16, 2, 128, "bf16", "e4m3", "hnd", 16),
    ([8, 1, 3], [500, 64, 65], 8, 1, 128, "f16", "e4m3", "nhd", 128),
    ([40, 30], [300, 30], 8, 2, 128, "bf16", "e4m3", "hnd", 32),
    ([8, 5], [900, 77], 16, 2, 64, "bf16", "e4m3", "nhd", 64),
    ([30, 2], [200, 1000], 16, 2, 64, "f16", "e4m3", "hnd", 16),
    ([2, 1], [333, 2000], 16, 2, 256, "f16", "e4m3", "hnd", 512),
    ([20, 1], [400, 100], 16, 2, 256, "bf16", "e4m3", "nhd", 16),
]


@pytest.mark.parametrize("new,length,hq,hkv,dim,kind,cache,layout,page", ATTEND_8BIT)
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 5)])
def test_attend_8_bit(new, length, hq, hkv, dim, kind, cache, layout, page, window, sinks):
    b = Batch(new, length, hq, hkv, dim, kind, cache, layout, page, seed=len(new) + dim)
    b.run(window, sinks)
    b.check(window, sinks)
    assert b.status.tolist() == [0] * len(new)


def test_attend_caches_inside_one_tensor_and_strided_output():
    """Keys and values of a page next to each other, and an output with gaps between its tokens."""
    kv = _kv()
    b = Batch([3, 1], [100, 40], 8, 2, 128, "bf16", "bf16", "nhd", 16)
    both = torch.full((b.pages, 2, 16, 2, 128), math.nan, dtype=torch.bfloat16, device="cuda")
    both[:, 0], both[:, 1] = b.kc, b.vc
    wide = torch.full((4, 8 * 128 + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    out = wide[:, :1024].view(4, 8, 128)
    kv.ss_attend(b.plan, b.q, both[:, 0], both[:, 1], b.table, _i32(b.length), b.cu, out=out, row_status=b.status, workspace=b.workspace,
                 scale=b.scale, lse=b.lse)
    b.out[:4] = out
    b.check()
    assert torch.all(wide[:, 1024:] == 7.0)


def test_far_pages_of_a_large_cache():
    """Pages whose offset passes 2^32 elements: stored by ss_rope_store and read by ss_attend there and nowhere else."""
    if torch.cuda.mem_get_info()[0] < 30 << 30:
        pytest.skip("needs 30 GB of free device memory")
    kv = _kv()
    page, hkv, dim, tokens = 64, 8, 128, 130
    pages = 2 ** 32 // (page * hkv * dim) + 4
    kc, vc = (torch.empty(pages, hkv, page, dim, dtype=torch.bfloat16, device="cuda").transpose(1, 2) for _ in range(2))
    mine = [pages - 1, 3, pages - 2]
    for p in mine:
        kc[p], vc[p] = math.nan, math.nan
    g = torch.Generator(device="cuda").manual_seed(9)
    q, k, v = (torch.randn(tokens, h, dim, generator=g, device="cuda").bfloat16() for h in (16, hkv, hkv))
    plan = _plan(1, tokens, page, pages, 3, q_heads=16, kv_heads=hkv, head_dim=dim, max_new=4)
    positions = torch.arange(tokens, device="cuda", dtype=torch.int32)
    slots = _i32([mine[t // page] * page + t % page for t in range(tokens)])
    assert int(slots.max()) * hkv * dim > 2 ** 32
    inv = torch.tensor(kv.rope_frequencies(dim), device="cuda")
    turned = torch.empty_like(q)
    kv.ss_rope_store(plan, q, k, v, kc, vc, inv, positions, slots, q_out=turned)
    out, status = torch.empty(4, 16, dim, dtype=torch.bfloat16, device="cuda"), _i32([0])
    workspace = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    kv.ss_attend(plan, turned[-4:], kc, vc, _i32([mine]), _i32([tokens]), _i32([0, 4]), out=out, row_status=status, workspace=workspace,
                 scale=dim ** -0.5)
    torch.cuda.synchronize()
    held_k = torch.stack([kc[mine[t // page], t % page] for t in range(tokens)])
    held_v = torch.stack([vc[mine[t // page], t % page] for t in range(tokens)])
    assert torch.equal(held_v, v)
    want = ref.rope(k, None, positions, inv, False)
    assert torch.all((held_k.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -16)
    want, _, weighted, _, _ = ref.attend(turned[-4:].double(), held_k.double(), held_v.double(), tokens - 4, dim ** -0.5)
    assert torch.all((out.double() - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2.0 ** -16) * weighted + 2.0 ** -20)
    assert status.tolist() == [0]


def test_guard_bands_around_what_is_written():
    """Outputs, log-sum-exps, workspace, slots, positions and tables sit between bands that must not change."""
    kv = _kv()
    guard = 4096

    def banded(shape, dtype, fill=0):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        raw = torch.full((n + 2 * guard,), 0xA5, dtype=torch.uint8, device="cuda")
        t = raw[guard:guard + n].view(dtype).view(shape)
        t.fill_(fill)
        bands.append((raw, n))
        return t

    bands = []
    b = Batch([5, 1, 9, 1], [700, 3, 9, 2500], 12, 2, 64, "f16", "f16", "hnd", 16)
    b.out, b.lse, b.status = banded((16, 12, 64), torch.float16), banded((16, 12), torch.float32), banded((4,), torch.int32)
    b.workspace = banded((b.plan.workspace_bytes,), torch.uint8)
    for window in (0, 33):
        b.run(window, 2)
    plan = _plan(3, 40, 16, 60, 5)
    table, slots, positions = banded((3, 5), torch.int32, -1), banded((40,), torch.int32), banded((40,), torch.int32)
    seq, status, kv_len = banded((3,), torch.int32), banded((3,), torch.int32), banded((3,), torch.int32)
    free, count = banded((60,), torch.int32), banded((1,), torch.int32, 60)
    free.copy_(torch.arange(60))
    for _ in range(2):
        kv.ss_kv_append(plan, table, kv_len, free, count, _i32([0, 20, 21, 40]), slots=slots, positions=positions, seq_len=seq, row_status=status)
        kv.ss_kv_commit(plan, table, kv_len, free, count, seq, counts=_i32([18, 0, 5]), finished=_i32([0, 0, 1]))
    cache = banded((2, 60, 2, 16, 64), torch.bfloat16)
    q = torch.randn(40, 4, 64, device="cuda").bfloat16()
    q_out = banded((40, 4, 64), torch.bfloat16)
    kv.ss_rope_store(plan, q, q[:, :2].contiguous(), q[:, 2:].contiguous(), cache[0].transpose(1, 2), cache[1].transpose(1, 2),
                     torch.tensor(kv.rope_frequencies(64), device="cuda"), positions, slots, q_out=q_out)
    torch.cuda.synchronize()
    for raw, n in bands:
        assert torch.all(raw[:guard] == 0xA5) and torch.all(raw[guard + n:] == 0xA5)


def test_attend_sharp_scores():
    """Scores of some hundreds: the running maximum moves, weights underflow."""
    b = Batch([3, 1], [900, 70], 8, 2, 128, "bf16", "bf16", "hnd", 16, spread=30.0)
    b.run()
    b.check()


def test_attend_queries_before_the_cache():
    """More new tokens than the row holds: the first queries see nothing and give zeros."""
    b = Batch([4, 2], [2, 0], 4, 2, 64, "bf16", "bf16", "hnd", 16)
    b.run()
    b.check()


@pytest.mark.parametrize("kind,cache,dim,hq", [("bf16", "bf16", 128, 8), ("f16", "f16", 64, 24), ("bf16", "e4m3", 128, 2),
                                               ("f16", "f16", 256, 8)])
def test_attend_values_that_are_not_finite_stay_with_who_sees_them(kind, cache, dim, hq):
    b = Batch([4, 1], [200, 90], hq, 2, dim, kind, cache, "hnd", 16)
    wild = math.nan if cache == "e4m3" else math.inf
    # the third new token of row 0, and a token of row 1 that has left its window
    for r, t in ((0, 198), (1, 5)):
        page, place = int(b.table[r, t // 16]), t % 16
        if cache == "e4m3":
            b.vc.view(torch.uint8)[page, place, 1, 7] = 0x7F
            b.kc.view(torch.uint8)[page, place, 1, 9] = 0x7F if r else b.kc.view(torch.uint8)[page, place, 1, 9]
        else:
            b.vc[page, place, 1, 7] = wild
            if r:
                b.kc[page, place, 1, 9] = math.nan
        b.v[r][t, 1, 7] = wild
    b.run(window=80)
    torch.cuda.synchronize()
    got, half = b.out[:5].double(), hq // 2
    # queries 2 and 3 of row 0 see it, in its head's column only
    expect = torch.zeros_like(got, dtype=torch.bool)
    expect[2:4, half:, 7] = True
    assert torch.equal(~torch.isfinite(got), expect)
    if cache != "e4m3":
        assert torch.all(got[2:4, half:, 7] == math.inf)
    b.v[0][198, 1, 7] = 0.0
    b.v[1][5, 1, 7] = 0.0
    b.k[1][5, 1, 9] = 0.0
    b.out[2:4, half:, 7] = 0.0
    want0 = ref.attend(b.q[:4].double(), b.k[0], b.v[0], 196, b.scale, 80)[0]
    keep = ~expect[:4]
    assert torch.all((got[:4] - want0).abs()[keep] <= (0.02 * (1 + want0.abs()))[keep])
    want1 = ref.attend(b.q[4:5].double(), b.k[1], b.v[1], 89, b.scale, 80)[0]
    assert torch.all((got[4:] - want1).abs() <= 0.02 * (1 + want1.abs()))


def test_attend_bad_pages_are_not_visible():
    b = Batch([2, 1, 1], [300, 100, 40], 8, 2, 128, "bf16", "bf16", "hnd", 16)
    hidden = {0: set(range(32, 48)) | set(range(160, 176)), 1: set(range(96, 100))}
    b.table[0, 2], b.table[0, 10], b.table[1, 6] = b.pages, -1, 2 ** 31 - 1
    b.run()
    b.check(hidden=hidden)
    assert b.status.tolist() == [1 << 13, 1 << 13, 0]
    b = Batch([2], [300], 8, 2, 128, "bf16", "bf16", "hnd", 64)
    b.table[0, 1] = -2 ** 31
    b.run()
    b.check(hidden={0: set(range(64, 128))})
    assert b.status.tolist() == [1 << 13]


def test_attend_bad_rows_are_reported():
    b = Batch([1, 2, 1], [30, 50, 20], 4, 2, 64, "bf16", "bf16", "hnd", 16)
    lengths = b.length
    b.length = [30, -1, 20]
    b.run()
    torch.cuda.synchronize()
    assert b.status.tolist() == [0, 1 << 4, 0]
    assert torch.all(b.out[1:3] == 0)
    b.length = [30, 2 ** 31 - 1, 20]
    b.status.zero_()
    b.run()
    torch.cuda.synchronize()
    assert b.status.tolist() == [0, 1 << 4, 0]
    b.length, b.cu = lengths, _i32([0, 1, 3, 900])
    b.status.zero_()
    b.out.fill_(7.0)
    b.run()
    torch.cuda.synchronize()
    assert b.status.tolist() == [0, 0, 1 << 9]
    assert torch.all(b.out[3] == 7.0) and torch.all(b.out[0] != 7.0)


def test_attend_on_another_stream_and_in_a_graph():
    b = Batch([2, 1, 5], [500, 40, 77], 8, 2, 128, "bf16", "bf16", "hnd", 16)
    lengths = _i32(b.length)
    args = dict(out=b.out[:8], row_status=b.status, workspace=b.workspace, scale=b.scale, lse=b.lse[:8])
    kv, side = _kv(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    kv.ss_attend(b.plan, b.q, b.kc, b.vc, b.table, lengths, b.cu, stream=side, **args)
    side.synchronize()
    b.check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.ss_attend(b.plan, b.q, b.kc, b.vc, b.table, lengths, b.cu, **args)
    for length in ([400, 13, 5], [500, 1, 77]):
        b.out[:8] = 7.0
        lengths.copy_(_i32(length))
        graph.replay()
        b.length = length
        for r, n in enumerate(length):
            b.k[r], b.v[r] = b.k[r][:max(n, 1)] if r != 1 else b.k[r][:n], b.v[r][:max(n, 1)] if r != 1 else b.v[r][:n]
        b.check()
        b2 = Batch([2, 1, 5], [500, 40, 77], 8, 2, 128, "bf16", "bf16", "hnd", 16)
        b.k, b.v = b2.k, b2.v


def test_attend_long_rows_are_split():
    """One long row over every CTA, beside rows of one token."""
    b = Batch([1, 2, 1], [1, 20000, 2], 4, 1, 128, "bf16", "bf16", "hnd", 64)
    b.run()
    torch.cuda.synchronize()
    got = b.out[1:3].double()
    q, k, v = b.q[1:3].double(), b.k[1][:, 0], b.v[1][:, 0]
    s = torch.einsum("nhd,td->nht", q, k) * b.scale
    s[0, :, 19999] = -math.inf
    w = torch.softmax(s, -1)
    want = torch.einsum("nht,td->nhd", w, v)
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -8 * torch.einsum("nht,td->nhd", w, v.abs()) * 1.01 + 2.0 ** -20
    assert torch.all((got - want).abs() <= tol)


# ------------------------------------------------------------------ prefix sums that pass the buffers
def test_append_leaves_out_rows_past_its_buffers():
    kv = _kv()
    plan = _plan(3, 40, 16, 60, 5)
    for entries in (40, 39, 20, 19, 0):
        room = _i32([99] * 2 * 64)
        slots, positions = room[:entries], room[64:64 + min(40, entries + 1)]
        seq, status = _i32([99] * 3), _i32([99] * 3)
        table = _i32([[-1] * 5] * 3)
        kv.ss_kv_append(plan, table, _i32([0, 0, 0]), _i32(list(range(60))), _i32([60]), _i32([0, 20, 21, 40]), slots=slots,
                        positions=positions, seq_len=seq, row_status=status)
        torch.cuda.synchronize()
        served = sum(t <= entries for t in (20, 21, 40))
        new = [20, 1, 19]
        assert status.tolist() == [0] * served + [1 << 4] * (3 - served)
        assert seq.tolist() == new[:served] + [0] * (3 - served)
        assert torch.all(room[entries:64] == 99) and torch.all(room[64 + entries:] == 99)
        tokens = sum(new[:served])
        assert torch.all(slots[:tokens] >= 0) and torch.all(slots[tokens:] == -1)


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_attend_leaves_out_rows_past_its_queries(cache):
    b = Batch([2, 1, 3], [500, 40, 77], 8, 2, 128, "bf16", cache, "hnd", 16)
    b.q = b.q[:4]
    b.run()
    torch.cuda.synchronize()
    assert b.status.tolist() == [0, 0, 1 << 9]
    assert torch.all(b.out[3:] == 7.0) and torch.all(b.lse[3:] == 7.0)
    got, got_lse = b.out[:3].clone(), b.lse[:3].clone()
    b.q = b.q[:0]  # nothing to do
    b.run()
    whole = Batch([2, 1, 3], [500, 40, 77], 8, 2, 128, "bf16", cache, "hnd", 16)
    whole.run()
    whole.check()
    assert torch.equal(b.out[:3], got)
    # another cut of the work: the same sums in another order, each within the bounds above (scores stay below 30)
    assert torch.all((got_lse - whole.lse[:3]).abs() <= 2.0 ** -12)
    assert torch.all((got.double() - whole.out[:3].double()).abs() <= 2.0 ** -7 * whole.out[:3].double().abs() + 2.0 ** -7)


# ------------------------------------------------------------------ refusals with a plan
def test_calls_refuse_wrong_arguments():
    from spec_verification_gb300 import native
    kv = _kv()
    b = Batch([1], [20], 4, 2, 64, "bf16", "bf16", "hnd", 16)
    base = dict(plan=b.plan, q=b.q, k_cache=b.kc, v_cache=b.vc, block_table=b.table, seq_len=_i32([20]), cu_new=b.cu, out=b.out[:1],
                row_status=b.status, workspace=b.workspace, scale=b.scale)

    def refused(code, call, **change):
        with pytest.raises(native.SSError) as e:
            call(**change)
        assert e.value.code == code, change

    attend = lambda **c: kv.ss_attend(**{**base, **c})  # noqa: E731
    refused(-1, attend, B=2, block_table=torch.cat([b.table, b.table]))
    refused(-1, attend, scale=0.0)
    refused(-1, attend, scale=math.nan)
    refused(-1, attend, window=-1)
    refused(-1, attend, sinks=-1)
    refused(-4, attend, workspace=b.workspace[:-256])
    refused(-2, attend, workspace=torch.zeros(b.plan.workspace_bytes + 256, dtype=torch.uint8, device="cuda")[16:])
    refused(-1, attend, q=b.q.half())
    refused(-1, attend, q=b.q[:, :2])
    refused(-1, attend, k_cache=b.kc.half(), v_cache=b.vc.half())
    refused(-1, attend, k_cache=b.kc[:-1], v_cache=b.vc[:-1])
    refused(-1, attend, block_table=b.table[:, :1])
    refused(-1, attend, seq_len=torch.tensor([20], device="cuda"))
    refused(-1, attend, k_scale=torch.ones(2, device="cuda"))
    wide = torch.zeros(2, 4 * 64 + 4, dtype=torch.bfloat16, device="cuda")
    refused(-2, attend, q=wide[:, :256].view(2, 4, 64))
    off = torch.zeros(1 + 4 * 64, dtype=torch.bfloat16, device="cuda")
    refused(-2, attend, q=off[1:].view(1, 4, 64))
    k, v = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    inv = torch.tensor(kv.rope_frequencies(64), device="cuda")
    rbase = dict(plan=b.plan, q=b.q, k=k, v=v, k_cache=b.kc, v_cache=b.vc, inv_freq=inv, positions=_i32([3]), slots=_i32([-1]), q_out=b.out[:1])
    rope = lambda **c: kv.ss_rope_store(**{**rbase, **c})  # noqa: E731
    refused(-3, rope, inv_freq=inv[:5])
    refused(-1, rope, inv_freq=inv.float())
    refused(-1, rope, eps=-1.0)
    refused(-1, rope, rope_scale=math.inf)
    refused(-1, rope, positions=_i32([3, 4]))
    two = torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda")
    many = dict(q=two, q_out=two, k=torch.cat([k, k]), v=torch.cat([v, v]), positions=_i32([1, 2]), slots=_i32([-1, -1]))
    refused(-1, rope, **many)  # more tokens than the plan's
    refused(-1, rope, k=k.half())
    none = dict(q=b.q[:0], q_out=b.out[:0], k=k[:0], v=v[:0], positions=_i32([]), slots=_i32([]))
    rope(**none)  # no tokens: nothing to do
    pool = dict(plan=b.plan, block_table=b.table, kv_len=_i32([20]), free_pages=_i32([0] * b.pages), free_count=_i32([0]))
    refused(-1, lambda **c: kv.ss_kv_commit(**{**pool, **c}), seq_len=_i32([20]), B=2)
    refused(-1, lambda **c: kv.ss_kv_commit(**{**pool, **c}), seq_len=_i32([20]).long())
    refused(-1, lambda **c: kv.ss_kv_commit(**{**pool, **c}), seq_len=_i32([20]), free_pages=_i32([0]))
    kv.ss_attend(**base)  # and the call itself is fine
    kv.ss_rope_store(**rbase)
    torch.cuda.synchronize()


def test_calls_refuse_host_tensors():
    """A host address never reaches a kernel: rope_frequencies' result, for one, is a host array."""
    from spec_verification_gb300 import native
    kv = _kv()
    b = Batch([1], [20], 4, 2, 64, "bf16", "e4m3", "hnd", 16)
    attend = dict(plan=b.plan, q=b.q, k_cache=b.kc, v_cache=b.vc, block_table=b.table, seq_len=_i32([20]), cu_new=b.cu, out=b.out[:1],
                  row_status=b.status, workspace=b.workspace, scale=b.scale, lse=b.lse, k_scale=b.ks, v_scale=b.vs)
    k = torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    weight = torch.ones(64, dtype=torch.bfloat16, device="cuda")
    rope = dict(plan=b.plan, q=b.q, k=k, v=k, k_cache=b.kc, v_cache=b.vc, inv_freq=torch.tensor(kv.rope_frequencies(64), device="cuda"),
                positions=_i32([3]), slots=_i32([-1]), q_out=b.out[:1], q_weight=weight, k_weight=weight, k_scale=b.ks, v_scale=b.vs)
    pool = dict(plan=b.plan, block_table=b.table, kv_len=_i32([20]), free_pages=_i32([0] * b.pages), free_count=_i32([0]), seq_len=_i32([20]))
    append = dict(pool, cu_new=_i32([0, 0]), slots=_i32([]), positions=_i32([]), row_status=_i32([0]))
    commit = dict(pool, counts=_i32([0]), finished=_i32([0]))
    for call, args in ((kv.ss_attend, attend), (kv.ss_rope_store, rope), (kv.ss_kv_append, append), (kv.ss_kv_commit, commit)):
        for name, value in args.items():
            if torch.is_tensor(value):
                with pytest.raises(native.SSError) as e:
                    call(**{**args, name: value.cpu()})
                assert e.value.code == -1 and "host" in str(e.value), name
        call(**args)
    with pytest.raises(native.SSError):
        kv.ss_attend(**{**attend, "scale": 3e38})  # finite, but not in powers of two
    torch.cuda.synchronize()
