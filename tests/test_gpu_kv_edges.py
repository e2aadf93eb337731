"""The KV-cache operators on the GPU where many units follow one another in a CTA, and at values on the edge of their
types; bounds as in tests/test_gpu_kv.py."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import kv_reference as ref  # noqa: E402
from tests.test_gpu_kv import TYPES, U, Batch, _cache, _i32, _kv, _plan  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _env():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from spec_verification_gb300 import build
    build.build()


def _counters(b):
    """Every counter word of a batch's workspace: 3 a CTA, then the pieces (2 a CTA, a row tile of outputs and sums)."""
    rows = b.plan_new * (b.hq // b.hkv)
    tile = next(t for t in (16, 32, 64, 128) if rows <= t or t == 128)
    up = lambda x: -(-x // 256) * 256  # noqa: E731
    ctas = [g for g in range(1, 2048) if up(12 * g) + up(8 * g * tile * b.dim) + up(32 * g * tile) == b.plan.workspace_bytes]
    assert len(ctas) == 1
    return b.workspace[:12 * ctas[0]].view(torch.int32)


def _many(rows, most, longest, hq, hkv, dim, kind, cache, layout, page, seed):
    rng = np.random.default_rng(seed)
    new = rng.integers(1, most + 1, rows)
    new[0] = most
    length = np.maximum(new, (longest * rng.random(rows) ** 2).astype(int) + 1)
    b = Batch(new.tolist(), length.tolist(), hq, hkv, dim, kind, cache, layout, page, seed=seed)
    b.hq, b.plan_new = hq, most
    return b, rng


MANY = [
    # rows, most new, longest, hq, hkv, dim, type, cache, layout, page
    (700, 1, 400, 16, 4, 128, "bf16", "bf16", "hnd", 16),
    (320, 4, 300, 8, 4, 256, "f16", "f16", "nhd", 16),
    (320, 3, 400, 16, 4, 64, "f16", "f16", "hnd", 32),
    (320, 8, 260, 16, 2, 128, "bf16", "bf16", "nhd", 16),
    (500, 2, 600, 8, 4, 128, "bf16", "e4m3", "hnd", 16),    # 16 query rows: converted in registers
    (320, 7, 260, 18, 2, 64, "f16", "e4m3", "nhd", 16),     # 64
    (200, 8, 260, 32, 4, 128, "bf16", "e4m3", "hnd", 32),   # 64
    (160, 16, 260, 16, 2, 128, "f16", "e4m3", "hnd", 16),   # 128
    (160, 4, 260, 8, 4, 256, "bf16", "e4m3", "nhd", 16),
]


@pytest.mark.parametrize("rows,most,longest,hq,hkv,dim,kind,cache,layout,page", MANY)
@pytest.mark.parametrize("window,sinks", [(0, 0), (90, 20)])
def test_bad_pages_of_some_of_many_rows(rows, most, longest, hq, hkv, dim, kind, cache, layout, page, window, sinks):
    """More units than CTAs, so a CTA's units follow one another: what is hidden in one must not be in its neighbours."""
    b, rng = _many(rows, most, longest, hq, hkv, dim, kind, cache, layout, page, seed=rows + dim + most)
    hidden = {}
    for r in rng.choice(rows, rows // 12, replace=False).tolist():
        for block in rng.choice(-(-b.length[r] // page), rng.integers(1, 4)).tolist():
            b.table[r, block] = int(rng.choice([b.pages, -1, 2 ** 31 - 1, -2 ** 31]))
            hidden.setdefault(r, set()).update(range(block * page, block * page + page))
    assert len(hidden) >= 10
    b.run(window, sinks)
    b.check(window, sinks, hidden=hidden)
    status = b.status.tolist()
    assert all(status[r] == 0 for r in range(rows) if r not in hidden)
    if not window:
        assert all(status[r] == 1 << 13 for r in hidden)
    assert int(_counters(b).abs().sum()) == 0


# ------------------------------------------------------------------ rotary store
@pytest.mark.parametrize("tokens", [9, 400, 2600])  # one, two and four tokens to a CTA
@pytest.mark.parametrize("dim,rot,inter,kind,cache", [(64, 64, False, "bf16", "bf16"), (128, 48, False, "bf16", "e4m3"),
                                                       (128, 0, False, "bf16", "bf16"), (256, 256, True, "bf16", "bf16"),
                                                       (128, 128, False, "f16", "f16"), (64, 32, True, "f16", "e4m3")])
def test_norms_of_heads_whose_squares_pass_32_bits(tokens, dim, rot, inter, kind, cache):
    """Against 64 bits: squares whose sum overflows or vanishes in 32, an infinite value (the others are 0), NaN."""
    kv = _kv()
    g = torch.Generator(device="cuda").manual_seed(tokens + dim)
    plan = _plan(1, tokens, 16, -(-tokens // 16), 1, q_heads=4, kv_heads=2, head_dim=dim, dtype=kind, cache_dtype=cache)
    q, k = (torch.randn(tokens, h, dim, generator=g, device="cuda") for h in (4, 2))
    for x in (q, k):
        if kind == "bf16":
            x[0] *= 1e25
            x[1, 0, 5], x[tokens - 1, 1, dim - 2] = 3e38, -2e20
            x[2, 1] = x[2, 1].sign() * 3e38
            x[3] *= 1e-25
            x[4, 0] *= 1e-37
        x[5, 1, 3], x[6, 0, dim - 1], x[7, 1, 0] = math.inf, -math.inf, math.nan
    q, k, v = q.to(TYPES[kind]), k.to(TYPES[kind]), torch.zeros(tokens, 2, dim, device="cuda", dtype=TYPES[kind])
    qw, kw = (1 + 0.3 * torch.randn(2, dim, generator=g, device="cuda")).to(TYPES[kind])
    positions, slots = (torch.arange(tokens, device="cuda", dtype=torch.int32) + 1), torch.arange(tokens, device="cuda", dtype=torch.int32)
    inv = torch.tensor(kv.rope_frequencies(rot), device="cuda") if rot else None
    kc, vc = (_cache(cache, "hnd", -(-tokens // 16), 16, 2, dim, 0.0) for _ in range(2))
    out = torch.empty_like(q)
    for eps in (0.0, 1e-6):
        kv.ss_rope_store(plan, q, k, v, kc, vc, inv, positions, slots, q_out=out, q_weight=qw, k_weight=kw, eps=eps, interleaved=inter)
        held = kc[slots.long() // 16, slots.long() % 16].double() if cache != "e4m3" else kc.double().reshape(-1, 2, dim)[:tokens]
        for got, x, w, low in ((out.double(), q, qw, False), (held, k, kw, cache == "e4m3")):
            want = ref.rope(x, w, positions, inv, inter, eps=eps)
            size = want.abs()
            if rot:
                a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
                size[..., a] = size[..., b] = size[..., a] + size[..., b]
            tol = (16 * 2.0 ** -24 + 2.0 ** -22) * 1.5 * size + 2.0 ** -25
            if low:
                want = want.clamp(-448, 448)
                tol = tol * (1 + U["e4m3"]) + 2.0 ** -10
            tol = tol + U["e4m3" if low else kind] * want.abs()
            assert torch.equal(torch.isnan(got), torch.isnan(want))
            assert torch.all(((got - want).abs() <= tol) | torch.isnan(want)), (eps, (got - want).abs().nan_to_num(0).max())
            assert torch.all(torch.isfinite(got[0]))


# ------------------------------------------------------------------ attention: weights and scores at the ends of their types
class Row:
    """One row over given keys and values [tokens, hkv, dim] in scattered pages, `times` times in a batch."""

    def __init__(self, q, k, v, kind, cache, page=64, k_scale=None, v_scale=None, times=1):
        kv = _kv()
        n, hq, self.dim = q.shape
        tokens, hkv = k.shape[:2]
        blocks = -(-tokens // page)
        g = torch.Generator(device="cuda").manual_seed(tokens)
        ids = torch.randperm(blocks + 2, generator=g, device="cuda")[:blocks]
        self.q, self.tokens, self.kind, self.product = q.to(TYPES[kind]).contiguous(), tokens, kind, "f16" if cache == "e4m3" else kind
        self.ks, self.vs, self.scale = k_scale, v_scale, self.dim ** -0.5

        def held(x, scale):
            y = (x if scale is None else (x / scale[:, None]).clamp(-448, 448)).to(TYPES[cache])
            full = torch.zeros(blocks * page, hkv, self.dim, dtype=y.dtype, device="cuda").view(torch.uint8)
            full[:tokens] = y.view(torch.uint8)
            c = _cache(cache, "nhd", blocks + 2, page, hkv, self.dim, math.nan)
            c.view(torch.uint8)[ids] = full.view(blocks, page, hkv, -1)
            return c, y.double() * (1.0 if scale is None else scale.double()[:, None])

        (self.kc, self.k), (self.vc, self.v) = held(k, k_scale), held(v, v_scale)
        self.plan = kv.Plan(max_rows=times, max_tokens=n * times, max_new=n, q_heads=hq, kv_heads=hkv, head_dim=self.dim, page_size=page,
                            num_pages=blocks + 2, max_blocks=blocks, dtype=kind, cache_dtype=cache)
        self.times, self.table, self.status = times, ids.to(torch.int32).repeat(times, 1), _i32([0] * times)
        self.workspace = torch.zeros(self.plan.workspace_bytes, dtype=torch.uint8, device="cuda")

    def run(self, **kw):
        """Outputs [times, n, hq, dim] and log-sum-exps."""
        n, hq, d = self.q.shape
        q = self.q.repeat(self.times, 1, 1)
        out, lse = torch.empty_like(q), torch.empty(n * self.times, hq, device="cuda")
        _kv().ss_attend(self.plan, q, self.kc, self.vc, self.table, _i32([self.tokens] * self.times), _i32(list(range(0, n * self.times + 1, n))),
                        out=out, row_status=self.status, workspace=self.workspace, scale=self.scale, lse=lse, k_scale=self.ks, v_scale=self.vs, **kw)
        torch.cuda.synchronize()
        assert self.status.tolist() == [0] * self.times
        return out.double().view(self.times, n, hq, d), lse.double().view(self.times, n, hq)


# query rows, columns, type, cache: every kernel whose weights are f16
F16_WEIGHTS = [(4, 64, "f16", "f16"), (64, 64, "f16", "f16"), (16, 128, "f16", "f16"), (128, 128, "f16", "f16"), (8, 256, "f16", "f16"),
               (4, 64, "bf16", "e4m3"), (16, 128, "f16", "e4m3"), (32, 128, "bf16", "e4m3"), (64, 128, "f16", "e4m3"),
               (128, 64, "bf16", "e4m3"), (8, 256, "bf16", "e4m3")]


@pytest.mark.parametrize("rows,dim,kind,cache", F16_WEIGHTS)
@pytest.mark.parametrize("times,first", [(1, 0), (80, 0), (80, 128 * 100)])
def test_faint_keys_beside_dominant_ones(rows, dim, kind, cache, times, first):
    """60000 keys at about 2^-25.7 of eight (one for every 16 keys of a tile): each weight is held to 2^-11 of itself or to
    2^-32 of the largest.  80 rows are enough that a CTA has some 60000 keys, one row is split over all CTAs."""
    g = torch.Generator(device="cuda").manual_seed(rows + dim)
    tokens, hkv, group = 60000, 4, 4
    n = rows // group
    factors = (0.02 + 0.02 * torch.rand(hkv, generator=g, device="cuda")) if cache == "e4m3" else None
    one = torch.randn(hkv, dim, generator=g, device="cuda")  # all queries of a key head
    q = one.repeat_interleave(group, 0).expand(n, hkv * group, dim)
    k = 0.01 * torch.randn(tokens, hkv, dim, generator=g, device="cuda")
    v = 1 + 0.1 * torch.randn(tokens, hkv, dim, generator=g, device="cuda")
    k[first:first + 128:16] = one * (17.8 * dim ** 0.5 / one.square().sum(-1, keepdim=True))
    v[first:first + 128:16] = 0.0
    row = Row(q, k, v, kind, cache, k_scale=factors, v_scale=factors, times=times)
    got, got_lse = row.run()
    want, lse, weighted, plain, size = ref.attend(row.q.double(), row.k, row.v, tokens - n, row.scale)
    assert 2e-5 < want.min() and want.max() < 1e-3
    off = (dim * 2.0 ** -23 * size + 2.0 ** -20)[..., None]
    tol = U[kind] * want.abs() * (1 + 2.0 ** -10) + (U["f16"] + 2 * off) * weighted + 2.0 ** -32 * plain * (1 + 2.0 ** -10) + 2.0 ** -25
    assert torch.all((got - want).abs() <= tol), ((got - want).abs() / tol).max().item()
    assert torch.all((got_lse - lse).abs() <= 2 * off[..., 0] + 2.0 ** -22 * lse.abs())


@pytest.mark.parametrize("rows,dim,kind", [(8, 64, "bf16"), (8, 128, "bf16"), (16, 128, "f16"), (24, 128, "bf16"), (64, 128, "bf16"),
                                           (128, 64, "bf16"), (64, 64, "f16"), (8, 256, "bf16")])
@pytest.mark.parametrize("factor", [3e-7, 1e-30, 2.0 ** -126])
def test_queries_of_zeros_and_small_factors_over_8_bits(rows, dim, kind, factor):
    """Every score is 0: the mean of the values that a query sees, in tiles that it sees in part too."""
    g = torch.Generator(device="cuda").manual_seed(rows + dim)
    tokens, hkv, group = 300, 2, 4
    n = rows // group
    q = torch.randn(n, hkv * group, dim, generator=g, device="cuda")
    q[:, 1::2] = 0.0
    k, v = torch.randn(2, tokens, hkv, dim, generator=g, device="cuda")
    ones = torch.ones(hkv, device="cuda")
    row = Row(q, k * factor, v, kind, "e4m3", k_scale=factor * ones, v_scale=ones)
    for kw in ({}, {"window": 40, "sinks": 3}):
        got, got_lse = row.run(**kw)
        want, lse, weighted, plain, _ = ref.attend(row.q.double(), row.k, row.v, tokens - n, row.scale, **kw)
        # scores and weights are exact, but for 2^x (2^-20) and what scores of 2^-12 are rounded to
        tol = U[kind] * want.abs() * (1 + 2.0 ** -10) + (U["f16"] + 2.0 ** -19) * weighted + 2.0 ** -25
        assert torch.all((got - want).abs() <= tol)
        assert torch.all((got_lse - lse).abs() <= 2.0 ** -18)


@pytest.mark.parametrize("cache,page", [("bf16", 16), ("e4m3", 64)])  # tiles of 64 and of 128 keys
def test_sinks_near_two_to_the_31(cache, page):
    """The largest table row there is, and as many first tokens visible: a window that hides nothing."""
    kv = _kv()
    b = Batch([3, 2], [300, 1000], 8, 2, 64, "bf16", cache, "hnd", page)
    blocks = (2 ** 31 - 1) // page
    b.plan = kv.Plan(max_rows=2, max_tokens=5, max_new=3, q_heads=8, kv_heads=2, head_dim=64, page_size=page, num_pages=b.pages,
                     max_blocks=blocks, dtype="bf16", cache_dtype=cache)
    b.workspace = torch.zeros(b.plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    table = torch.empty(2, blocks, dtype=torch.int32, device="cuda")
    table[:, :b.table.shape[1]] = b.table
    b.table = table
    for sinks in (2 ** 31 - 1, blocks * page - 1, 2 ** 30):
        b.run(window=70, sinks=sinks)
        b.check()
    assert b.status.tolist() == [0, 0]


def test_one_token_of_any_stride():
    """One token taken out of rows of an odd length: its stride is of no matter."""
    kv = _kv()
    b = Batch([1], [70], 8, 2, 64, "bf16", "bf16", "hnd", 16)
    wide, out = (torch.zeros(3, 8 * 64 + 5, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    wide[0, :512] = b.q[0].flatten()
    b.q = wide[:1, :512].view(1, 8, 64)
    held, b.out = b.out, out[:1, :512].view(1, 8, 64)
    b.run()
    held[:1] = b.out
    b.out = held
    b.check()
    assert torch.all(out[:, 512:] == 0) and torch.all(out[1:] == 0)
    # an unaligned address is still refused
    from spec_verification_gb300 import native
    with pytest.raises(native.SSError) as e:
        b.q = wide[:1, 1:513].view(1, 8, 64)
        b.run()
    assert e.value.code == -2


# ------------------------------------------------------------------ attention: forms of the kernels that other tests do not reach
@pytest.mark.parametrize("hq,new,dim,kind", [(16, 4, 128, "bf16"), (16, 8, 128, "f16"), (16, 16, 128, "bf16"), (16, 4, 64, "bf16"),
                                             (16, 8, 64, "f16"), (24, 16, 64, "bf16"), (8, 2, 256, "f16"), (16, 16, 256, "bf16")])
@pytest.mark.parametrize("window,sinks", [(0, 0), (80, 5)])
def test_values_that_are_not_finite_over_8_bits(hq, new, dim, kind, window, sinks):
    """NaN in a value that some queries see, and in keys and values that none does: the converting kernels."""
    b = Batch([new, 1, 1], [200, 90, 300], hq, 2, dim, kind, "e4m3", "hnd", 16)
    nan = 0x7F
    where = [(0, 200 - new // 2, 1, 7)] + ([(1, 6, 0, 9), (2, 130, 1, dim - 1)] if window else [])
    for r, t, h, d in where:
        page, place = int(b.table[r, t // 16]), t % 16
        b.vc.view(torch.uint8)[page, place, h, d] = nan
        if r:
            b.kc.view(torch.uint8)[page, place, h, d] = nan
    b.run(window, sinks)
    torch.cuda.synchronize()
    half = hq // 2
    wild = torch.zeros(new + 2, hq, dim, dtype=torch.bool, device="cuda")
    wild[new - new // 2:new, half:, 7] = True  # the queries from that token on, in its head's column
    got = b.out[:new + 2]
    assert torch.equal(torch.isnan(got), wild)
    b.v[0][200 - new // 2, 1, 7] = 0.0
    at = 0
    for r, n in enumerate(b.new):
        want, _, weighted, plain, size = ref.attend(b.q[at:at + n].double(), b.k[r], b.v[r], b.length[r] - n, b.scale, window, sinks)
        off = (dim * 2.0 ** -23 * size + 2.0 ** -20)[..., None]
        tol = U[kind] * want.abs() * (1 + 2.0 ** -10) + (U["f16"] + 2 * off) * weighted + 2.0 ** -25 + 2.0 ** -32 * plain
        assert torch.all(((got[at:at + n].double() - want).abs() <= tol) | wild[at:at + n])
        at += n


@pytest.mark.parametrize("hq,hkv,kind,cache,page", [(4, 1, "bf16", "bf16", 16), (2, 2, "f16", "e4m3", 16), (24, 1, "bf16", "e4m3", 32)])
def test_as_many_rows_as_a_plan_may_have(hq, hkv, kind, cache, page):
    """8192 rows, each thread of the search for a CTA's range holds many; some rows are bad, some have nothing new."""
    rows, dim = 8192, 64
    rng = np.random.default_rng(hq)
    new = (rng.random(rows) < 0.9).astype(int)
    length = 1 + (rng.random(rows) ** 4 * 60).astype(int)
    length[rng.integers(0, rows, 4)] = 3000
    b = Batch([1] * 2, [1] * 2, hq, hkv, dim, kind, cache, "hnd", page)  # types, factors
    g = torch.Generator(device="cuda").manual_seed(hq)
    used = -(-length // page)
    blocks, pages = int(used.max()), int(used.sum())
    first = np.cumsum(used) - used
    table = torch.full((rows, blocks), -1, dtype=torch.int32)
    ids = torch.randperm(pages, generator=g, device="cuda")
    for r in range(rows):
        table[r, :used[r]] = torch.arange(first[r], first[r] + used[r])
    table = torch.where(table.cuda() >= 0, ids[table.cuda().clamp(min=0).long()].to(torch.int32), -1).contiguous()
    kc, vc = (torch.randn(pages, hkv, page, dim, generator=g, device="cuda").to(TYPES[cache]).transpose(1, 2) for _ in range(2))
    q = torch.randn(int(new.sum()), hq, dim, generator=g, device="cuda").to(TYPES[kind])
    seq = length.copy()
    bad = rng.choice(rows, 20, replace=False)
    seq[bad] = -1
    plan = _kv().Plan(max_rows=rows, max_tokens=rows, max_new=1, q_heads=hq, kv_heads=hkv, head_dim=dim, page_size=page, num_pages=pages,
                      max_blocks=blocks, dtype=kind, cache_dtype=cache)
    out, status = torch.full_like(q, 7.0), _i32([0] * rows)
    workspace = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    _kv().ss_attend(plan, q, kc, vc, table, _i32(seq.tolist()), _i32([0] + np.cumsum(new).tolist()), out=out, row_status=status,
                    workspace=workspace, scale=dim ** -0.5, k_scale=b.ks, v_scale=b.vs)
    torch.cuda.synchronize()
    want_status = np.zeros(rows, int)
    want_status[bad] = 1 << 4
    assert status.tolist() == want_status.tolist()
    at = np.cumsum(new) - new
    for some in (np.flatnonzero((new > 0) & (seq > 0))[::7], np.flatnonzero((new > 0) & (seq >= 3000))):
        for r in some.tolist():
            t = torch.arange(int(seq[r]), device="cuda")
            k, v = (c[table[r, t // page].long(), t % page].double() if cache != "e4m3" else
                    c.view(torch.uint8)[table[r, t // page].long(), t % page].view(TYPES[cache]).double() for c in (kc, vc))
            if cache == "e4m3":
                k, v = k * b.ks.double()[:, None], v * b.vs.double()[:, None]
            k, v = (x.repeat_interleave(hq // hkv, 1) for x in (k, v))
            w = torch.softmax(torch.einsum("hd,thd->ht", q[at[r]].double(), k) * dim ** -0.5, -1)
            want, weighted = torch.einsum("ht,thd->hd", w, v), torch.einsum("ht,thd->hd", w, v.abs())
            product = U["f16" if cache == "e4m3" else kind]
            # 2^-14: 64 roundings of sums of |q k| below 16, twice, and the 2^x
            tol = U[kind] * want.abs() * (1 + 2.0 ** -10) + (product + 2.0 ** -14) * weighted + 2.0 ** -24
            assert torch.all((out[at[r]].double() - want).abs() <= tol), r
    for r in bad.tolist():
        if new[r]:
            assert torch.all(out[at[r]] == 0)


@pytest.mark.parametrize("wrong", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("inter", [False, True])
def test_frequencies_that_are_not_finite_show(wrong, inter):
    """The pairs of such a frequency become NaN, not what they were; the others are as they should be."""
    kv = _kv()
    plan = _plan(1, 5, 16, 1, 1, q_heads=2, kv_heads=1, head_dim=64)
    q, k, v = (torch.randn(5, h, 64, device="cuda").bfloat16() for h in (2, 1, 1))
    kc, vc = _cache("bf16", "hnd", 1, 16, 1, 64, 0.0), _cache("bf16", "hnd", 1, 16, 1, 64, 0.0)
    good = torch.tensor(kv.rope_frequencies(32), device="cuda")
    inv = good.clone()
    inv[3] = wrong
    places = torch.arange(5, device="cuda", dtype=torch.int32)
    outs = []
    for f in (good, inv):
        outs.append(torch.empty_like(q))
        kv.ss_rope_store(plan, q, k, v, kc, vc, f, places, places, q_out=outs[-1], interleaved=inter)
    torch.cuda.synchronize()
    nan = torch.zeros(64, dtype=torch.bool, device="cuda")
    nan[[6, 7] if inter else [3, 19]] = True
    assert torch.equal(torch.isnan(outs[1]), nan.expand_as(q)) and torch.equal(torch.isnan(kc[0, :5, 0]), nan.expand(5, 64))
    assert torch.equal(outs[0][..., ~nan], outs[1][..., ~nan]) and torch.equal(vc[0, :5], v)


def _largest_score_wins(row, group, kind):
    """A query's output is the value of its largest score, wherever 32 bits tell which that is."""
    n, hq, dim = row.q.shape
    tokens = row.tokens
    for kw in ({}, {"window": 700, "sinks": 5}):
        got, got_lse = row.run(**kw)
        assert torch.all(torch.isfinite(got)) and torch.all(torch.isfinite(got_lse))
        t, p = torch.arange(tokens, device="cuda"), torch.arange(tokens - n, tokens, device="cuda")[:, None]
        seen = (t <= p) & ((t > p - kw["window"]) | (t < kw["sinks"]) if kw else torch.ones_like(t, dtype=torch.bool))
        kk, vv = row.k.repeat_interleave(group, 1), row.v.repeat_interleave(group, 1)
        s = torch.einsum("nhd,thd->nht", row.q.double(), kk) * row.scale
        size = torch.einsum("nhd,thd->nht", row.q.double().abs(), kk.abs()).amax(-1) * row.scale
        top, at = s.masked_fill(~seen[:, None], -math.inf).topk(2, -1)
        off = dim * 2.0 ** -23 * size  # of a score
        sure = top[..., 0] - top[..., 1] > 2 * off + 60
        assert sure.double().mean() > 0.9
        want = torch.stack([vv[at[..., 0][:, h], h] for h in range(hq)], 1)
        # the bound of tests/test_gpu_kv.py where one weight is all there is: the output's rounding and the weight's (the others'
        # are below 2^-80, whatever the scores are off by); log-sum-exp: the score, rounded with the factors
        tol = U[kind] * want.abs() * (1 + 2.0 ** -10) + U[row.product] * want.abs() + 2.0 ** -25
        assert torch.all(((got - want).abs() <= tol)[:, sure])
        assert torch.all(((got_lse - top[..., 0]).abs() <= off + 2.0 ** -21 * top[..., 0].abs())[:, sure])


@pytest.mark.parametrize("rows,dim,kind,cache,spread", [
    (rows, dim, kind, cache, s) for rows, dim, kind, cache in F16_WEIGHTS + [(4, 64, "bf16", "bf16"), (16, 128, "bf16", "bf16"),
                                                                              (64, 64, "bf16", "bf16"), (128, 256, "bf16", "bf16")]
    for s in (1e4, 3e7, 1e9 if kind == "f16" else 1e12, *([1e30] if kind == "bf16" else []))])
@pytest.mark.parametrize("times", [1, 60])
def test_scores_of_any_size(rows, dim, kind, cache, spread, times):
    """Scores spread by up to 1e30: a query's output is the value of its largest score, as far as 32 bits tell which that is."""
    g = torch.Generator(device="cuda").manual_seed(rows + dim)
    tokens, hkv, group = 1500, 4, 4
    n = rows // group
    a = min(spread ** 0.5, 1e4) if kind == "f16" else spread ** 0.5
    if cache == "f16" and spread > 1e8:
        spread = 1e8
    factors = torch.full((hkv,), spread / a / 50, device="cuda") if cache == "e4m3" else None
    q = a * torch.randn(n, hkv * group, dim, generator=g, device="cuda")
    k, v = torch.randn(2, tokens, hkv, dim, generator=g, device="cuda")
    row = Row(q, k * (spread / a), v, kind, cache, k_scale=factors, v_scale=torch.ones(hkv, device="cuda") if cache == "e4m3" else None, times=times)
    _largest_score_wins(row, group, kind)


@pytest.mark.parametrize("rows,dim", [(4, 64), (16, 128), (32, 128), (64, 64), (128, 128), (8, 256)])
def test_largest_bf16_queries_over_8_bits(rows, dim):
    """Queries of 3e37: they become f16 by a power of two, however large they are."""
    g = torch.Generator(device="cuda").manual_seed(rows + dim)
    tokens, hkv, group = 900, 4, 4
    q = 3e37 * torch.randn(rows // group, hkv * group, dim, generator=g, device="cuda").clamp(-5, 5)
    q[:, 1] *= 1e-37
    k, v = torch.randn(2, tokens, hkv, dim, generator=g, device="cuda")
    row = Row(q, k * 1e-4, v, "bf16", "e4m3", k_scale=torch.full((hkv,), 2e-6, device="cuda"), v_scale=torch.ones(hkv, device="cuda"))
    assert 2.0 ** 124 < row.q.abs().max() < math.inf
    got = row.run()[0][0]
    assert torch.all(torch.isfinite(got))
    small = ref.attend(row.q[:, 1:2].double(), row.k[:, :1], row.v[:, :1], tokens - rows // group, row.scale)[0][:, 0]
    assert torch.all((got[:, 1] - small).abs() <= 2.0 ** -7 * (small.abs() + row.v.abs().mean()))
    row.q = torch.cat([row.q[:, :1], row.q[:, 2:3], row.q[:, 2:]], 1).contiguous()
    _largest_score_wins(row, group, "bf16")
