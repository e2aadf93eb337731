"""The 8-bit cache with a factor for each block of tokens and head on the GPU, against plain forms in 64 bits
(tests/kv_blocks_reference.py, tests/kv_reference.py).

Bounds.  Factors are powers of two, so a quotient is exact and a value is rounded once: stores are compared bit for
bit, and so are loads (a product with a power of two, rounded once).  Attention: as for a cache with a factor for each
head (tests/test_gpu_kv.py), with these changes.  A weight times its values' factor, u, is rounded to f16: half a step
of it, or 2^-25 where it is below 2^-14; the largest u of a row is at least 2^6 (m is 7 below the first tile's largest), so the
latter is 2^-31 of the largest.  log2 of a factor less m is rounded to 2^-19 at most here (numbers up to 2^6), 2^-20 of a
weight, as is 2^x.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests import kv_blocks_reference as bref  # noqa: E402
from tests import kv_reference as ref  # noqa: E402

pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
U = {"bf16": 2.0 ** -8, "f16": 2.0 ** -11}
E4M3 = torch.float8_e4m3fn


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


def _bytes(layout, pages, page, heads, dim, fill=0x5A):
    shape = (pages, heads, page, dim) if layout == "hnd" else (pages, page, heads, dim)
    t = torch.full(shape, fill, dtype=torch.uint8, device="cuda").view(E4M3)
    return t.transpose(1, 2) if layout == "hnd" else t


class Store:
    """Rows whose pages are scattered over a cache, and what the cache should hold."""

    def __init__(self, rows, longest, hkv, dim, kind, layout, page, block, seed=0, spare=2):
        self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.rows, self.hkv, self.dim, self.kind, self.page, self.block = rows, hkv, dim, kind, page, block
        blocks = -(-longest // page)
        self.pages = rows * blocks + spare
        self.table = torch.randperm(self.pages, generator=self.g, device="cuda")[:rows * blocks].view(rows, blocks).to(torch.int32)
        self.cache = [_bytes(layout, self.pages, page, hkv, dim) for _ in range(2)]
        self.factor = [torch.full((self.pages, hkv, page // block), math.nan, device="cuda") for _ in range(2)]
        self.plan = _kv().Plan(max_rows=rows, max_tokens=rows * longest, q_heads=hkv, kv_heads=hkv, head_dim=dim, page_size=page,
                               num_pages=self.pages, max_blocks=blocks, dtype=kind, cache_dtype="e4m3")
        self.status = _i32([0] * rows)
        # what is held: [row][keys, values][head] -> (tokens of the row in units of their factors, factors)
        start = bref.decoded(torch.tensor([0x5A])).item()
        self.want = [[[(torch.full((blocks * page, dim), start, dtype=torch.float64), [math.nan] * (blocks * page // block)) for _ in range(hkv)]
                      for _ in range(2)] for _ in range(rows)]

    def values(self, new, size=1.0):
        t = sum(new)
        wide = torch.randn(max(1, t), 2 * self.hkv * self.dim + 8, generator=self.g, device="cuda") * size
        wide = (wide * torch.exp2(torch.randint(-3, 4, (max(1, t), 1), generator=self.g, device="cuda").float())).to(TYPES[self.kind])
        n = self.hkv * self.dim
        return wide[:t, :n].view(t, self.hkv, self.dim), wide[:t, n:2 * n].view(t, self.hkv, self.dim)

    def call(self, k, v, held, new, seq=None, cu=None, stream=None):
        seq = [h + n for h, n in zip(held, new)] if seq is None else seq
        cu = [0] + np.cumsum(new).tolist() if cu is None else cu
        _kv().ss_kv_store_blocks(self.plan, k, v, *self.cache, *self.factor, self.table, _i32(held), _i32(seq), _i32(cu), row_status=self.status,
                                 stream=stream)

    def expect(self, k, v, held, new, skip=()):
        at = 0
        for r, n in enumerate(new):
            for x, side in zip((k, v), self.want[r]):
                for h in range(self.hkv):
                    if n and r not in skip:
                        bref.store(*side[h], x[at:at + n, h].double().cpu(), held[r], self.block)
            at += n

    def check(self):
        torch.cuda.synchronize()
        for c, f, which in zip(self.cache, self.factor, range(2)):
            got = bref.decoded(c.view(torch.uint8).cpu())
            want = torch.full_like(got, bref.decoded(torch.tensor([0x5A])).item())
            want_f = torch.full(f.shape, math.nan)
            table = self.table.cpu().long()
            for r in range(self.rows):
                for h in range(self.hkv):
                    units, factors = self.want[r][which][h]
                    want[table[r], :, h] = units.view(-1, self.page, self.dim)
                    want_f[table[r], h] = torch.tensor(factors).view(-1, self.page // self.block)
            assert torch.equal(f.cpu().nan_to_num(-1.0), want_f.nan_to_num(-1.0))
            assert torch.equal(got.nan_to_num(1e4), want.nan_to_num(1e4))


STORES = [
    # held, new, heads, dim, type, layout, page, block
    ([0], [1], 1, 64, "bf16", "hnd", 16, 16),
    ([15, 16, 17, 0, 31], [1, 1, 1, 5, 2], 2, 128, "bf16", "hnd", 16, 16),
    ([5, 40, 16, 0], [3, 100, 0, 20], 3, 64, "f16", "nhd", 32, 16),
    ([7, 0, 63], [70, 130, 1], 2, 256, "bf16", "nhd", 64, 32),
    ([100, 0], [1, 300], 1, 128, "f16", "hnd", 128, 128),
    ([1, 0, 900], [1000, 5, 130], 1, 64, "bf16", "hnd", 1024, 1024),
    ([3] * 150, [1 + i % 4 for i in range(150)], 2, 64, "bf16", "hnd", 16, 16),  # more rows than a CTA's threads
]


@pytest.mark.parametrize("held,new,hkv,dim,kind,layout,page,block", STORES)
def test_store_and_load(held, new, hkv, dim, kind, layout, page, block):
    """What is held before comes from a first call, a second goes on with larger values, a third with some of them taken back."""
    kv = _kv()
    s = Store(len(held), max(h + n for h, n in zip(held, new)) + 8, hkv, dim, kind, layout, page, block, seed=dim + len(held))
    steps = [([0] * len(held), held, 0.5), (held, new, 3.0), ([h + n // 2 for h, n in zip(held, new)], [4] * len(held), 0.1)]
    for before, count, size in steps:
        k, v = s.values(count, size)
        s.call(k, v, before, count)
        s.expect(k, v, before, count)
        s.check()
    assert s.status.tolist() == [0] * len(held)
    # back: some slots twice, some outside the cache
    tokens = [(r, t) for r in range(len(held)) for t in range(before[r] + 4)][:400]
    tokens += tokens[:3]
    slots = [int(s.table[r, t // page]) * page + t % page for r, t in tokens]
    bad = [-1, s.pages * page, 2 ** 31 - 1, -2 ** 31]
    wide = torch.full((len(slots) + 5, 2 * hkv * dim), 7.0, device="cuda").to(TYPES[kind])
    k_out, v_out = (wide[:-1, i * hkv * dim:(i + 1) * hkv * dim].view(-1, hkv, dim) for i in range(2))
    kv.ss_kv_load_blocks(s.plan, *s.cache, *s.factor, _i32(slots + bad), k_out=k_out, v_out=v_out)
    torch.cuda.synchronize()
    assert torch.all(wide[-1] == 7.0)
    for which, out in enumerate((k_out, v_out)):
        want = torch.stack([torch.stack([s.want[r][which][h][0][t] * s.want[r][which][h][1][t // block] for h in range(hkv)]) for r, t in tokens])
        assert torch.equal(out[:len(slots)].cpu(), want.to(TYPES[kind])) and torch.all(out[len(slots):] == 0)


@pytest.mark.parametrize("kind", ["bf16", "f16"])
def test_store_of_special_values(kind):
    """Infinities, NaN, zeros, the ends of the factors' range, and factors that no store wrote."""
    s = Store(1, 64, 2, 64, kind, "hnd", 16, 16)
    x = torch.zeros(40, 2, 64, dtype=TYPES[kind], device="cuda")
    x[0, 0, :4] = torch.tensor([math.inf, -math.inf, math.nan, 3.0])
    x[1, 0, 5] = 448.0
    x[16, 0, :3] = torch.tensor([449.0, 464.0, -0.0])       # the next factor
    x[20, 1, 0] = torch.finfo(TYPES[kind]).max              # beyond the largest factor in bf16
    x[33, 0, 1] = torch.finfo(TYPES[kind]).tiny             # below the smallest in bf16
    x[34, 1, :] = math.nan                                  # nothing finite
    y = torch.randn(40, 2, 64, device="cuda").to(TYPES[kind])
    y[:, :, 3] = math.inf
    s.call(x, y, [0], [40])
    s.expect(x, y, [0], [40])
    s.check()
    # the block that starts at 32 goes on with a factor that is no power of two, one that is none at all, one past the range
    for factor in (3.0, math.nan, -1.0, 1e30, 0.0):
        for which in range(2):
            s.factor[which][int(s.table[0, 2]), :, 0] = factor
            for h in range(2):
                s.want[0][which][h][1][2] = factor
        z = (torch.randn(1, 2, 64, device="cuda") * 5).to(TYPES[kind])
        s.call(z, -z, [40], [1])
        s.expect(z, -z, [40], [1])
        s.check()


def test_store_leaves_out_rows_that_are_not_served():
    s = Store(6, 48, 1, 64, "bf16", "nhd", 16, 16)
    k, v = s.values([6] * 6)
    held, new = [3, 0, 10, 5, 0, 2], [6] * 6
    s.call(k, v, [0] * 6, held)
    s.expect(k, v, [0] * 6, held)
    s.check()
    table = s.table.clone()
    k, v = s.values(new)
    s.table[3, 0], s.table[4, 0] = s.pages, -5
    # row 1: the append served none of it; row 2: a length past its table row; rows 3 and 4: bad pages; row 5 goes past tokens
    s.call(k, v, held, new, seq=[9, 0, 2 ** 30, 11, 6, 8], cu=[0, 6, 12, 18, 24, 30, 37])
    s.expect(k, v, held, new, skip=(1, 2, 3, 4, 5))
    s.table = table
    s.check()
    assert s.status.tolist() == [0, 0, 1 << 4, 1 << 13, 1 << 13, 1 << 9]
    s.status.zero_()
    s.call(k, v, [9, -1, 10, 5, 0, 2], new, cu=[0, 6, 12, 11, 17, 23, 23], seq=[15, 5, 16, 11, 6, 2])
    at, wanted = [0, 6, 12, 11, 17, 23], {0: 9, 3: 5, 4: 0}
    for r, h in wanted.items():
        for x, side in zip((k, v), s.want[r]):
            bref.store(*side[0], x[at[r]:at[r] + 6, 0].double().cpu(), h, 16)
    s.check()
    assert s.status.tolist() == [0, 1 << 4, 1 << 9, 0, 0, 0]


def test_store_on_another_stream_and_in_a_graph():
    kv = _kv()
    s = Store(3, 64, 2, 128, "bf16", "hnd", 32, 16)
    k, v = s.values([20, 3, 1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s.call(k, v, [0, 0, 0], [20, 3, 1], stream=side)
    side.synchronize()
    s.expect(k, v, [0, 0, 0], [20, 3, 1])
    s.check()
    held, seq, cu = _i32([20, 3, 1]), _i32([22, 3, 5]), _i32([0, 2, 2, 6])
    k, v = s.values([10])
    k, v = k.contiguous(), v.contiguous()
    out = torch.empty(2, 6, 2, 128, dtype=torch.bfloat16, device="cuda")
    slots = _i32([0] * 6)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.ss_kv_store_blocks(s.plan, k, v, *s.cache, *s.factor, s.table, held, seq, cu, row_status=s.status)
        kv.ss_kv_load_blocks(s.plan, *s.cache, *s.factor, slots, k_out=out[0], v_out=out[1])
    for before, new in (([20, 3, 1], [2, 0, 4]), ([22, 3, 5], [0, 6, 1])):
        a, b = s.values([10], 4.0)
        k.copy_(a)
        v.copy_(b)
        held.copy_(_i32(before))
        seq.copy_(_i32([h + n for h, n in zip(before, new)]))
        cu.copy_(_i32([0] + np.cumsum(new).tolist()))
        tokens = [(r, h + j) for r, (h, n) in enumerate(zip(before, new)) for j in range(n)][:6]
        slots.copy_(_i32(([int(s.table[r, t // 32]) * 32 + t % 32 for r, t in tokens] + [-1] * 6)[:6]))
        graph.replay()
        s.expect(k, v, before, new)
        s.check()
        for i, (r, t) in enumerate(tokens):
            for which in range(2):
                want = torch.stack([s.want[r][which][h][0][t] * s.want[r][which][h][1][t // 16] for h in range(2)]).to(torch.bfloat16)
                assert torch.equal(out[which, i].cpu(), want)


# ------------------------------------------------------------------ attention
class Blocks:
    """Rows with their own keys and values over the pages of a cache whose other bytes are NaN and whose other factors are not
    numbers to compute with.  `spread`: factors are 2^(-spread .. spread); exact=False: the memory has larger numbers, of which
    the power of two counts."""

    def __init__(self, new, length, hq, hkv, dim, kind, layout, page, block, seed=0, spread=3, exact=True, size=1.5):
        kv = _kv()
        g = torch.Generator(device="cuda").manual_seed(seed)
        rows = len(new)
        blocks = max(1, max(-(-n // page) for n in length))
        used = [-(-n // page) for n in length]
        self.pages = sum(used) + 3
        ids = torch.randperm(self.pages, generator=g, device="cuda").tolist()
        self.scale, self.kind, self.dim, self.page = dim ** -0.5, kind, dim, page
        self.cache = [_bytes(layout, self.pages, page, hkv, dim, 0x7F) for _ in range(2)]
        odd = torch.tensor([math.nan, math.inf, -math.inf, 0.0, -3.0, 1e38, 1e-38], device="cuda")
        shape = (self.pages, hkv, page // block)
        self.factor = [odd[torch.randint(0, 7, shape, generator=g, device="cuda")] for _ in range(2)]
        table = torch.full((rows, blocks), -1, dtype=torch.int32)
        self.held, at = ([], []), 0
        for r, n in enumerate(length):
            mine = ids[at:at + used[r]]
            at += used[r]
            table[r, :used[r]] = torch.tensor(mine, dtype=torch.int32)
            token = torch.arange(n, device="cuda")
            where = torch.tensor(mine + [0], device="cuda")[token // page]
            for which in range(2):
                wide = spread if which else min(spread, 3)  # (of keys less: it goes into the scores)
                e = torch.rand(-(-max(n, 1) // block), hkv, generator=g, device="cuda") * 2 * wide - wide
                f = torch.exp2(e.round())
                bits = torch.randn(n, hkv, dim, generator=g, device="cuda").to(E4M3)
                self.cache[which].view(torch.uint8)[where, token % page] = bits.view(torch.uint8)
                self.factor[which][where, :, token % page // block] = f[token // block] * (1.0 if exact else 1.75)
                self.held[which].append(bits.double() * f[token // block].double()[..., None])
        self.table, self.new, self.length = table.cuda(), new, length
        self.tokens = sum(new)
        wide = (torch.randn(max(1, self.tokens), hq * dim + 16, generator=g, device="cuda") * size).to(TYPES[kind])
        self.q = wide[:, :hq * dim].view(-1, hq, dim)
        self.cu = _i32([0] + np.cumsum(new).tolist())
        self.out = torch.full((self.tokens + 1, hq, dim), 7.0, device="cuda").to(TYPES[kind])
        self.lse = torch.full((self.tokens + 1, hq), 7.0, device="cuda")
        self.status = _i32([0] * rows)
        self.plan = kv.Plan(max_rows=rows, max_tokens=max(1, self.tokens), max_new=max(1, max(new)), q_heads=hq, kv_heads=hkv, head_dim=dim,
                            page_size=page, num_pages=self.pages, max_blocks=blocks, dtype=kind, cache_dtype="e4m3")
        self.workspace = torch.zeros(self.plan.workspace_bytes, dtype=torch.uint8, device="cuda")

    def run(self, window=0, sinks=0, **kw):
        _kv().ss_attend_blocks(self.plan, self.q, *self.cache, *self.factor, self.table, _i32(self.length), self.cu, out=self.out,
                               row_status=self.status, workspace=self.workspace, scale=self.scale, window=window, sinks=sinks, lse=self.lse, **kw)

    def check(self, window=0, sinks=0, hidden=None):
        torch.cuda.synchronize()
        n, at = self.tokens, 0
        assert torch.all(self.out[n:] == 7.0) and torch.all(self.lse[n:] == 7.0)
        for r, m in enumerate(self.new):
            k, v = self.held[0][r], self.held[1][r]
            want, lse, weighted, _, size = ref.attend(self.q[at:at + m].double(), k, v, self.length[r] - m, self.scale, window, sinks,
                                                      None if hidden is None else hidden.get(r))
            got, got_lse = self.out[at:at + m].double(), self.lse[at:at + m].double()
            off = self.dim * 2.0 ** -23 * size + 2.0 ** -20  # of a weight, relative
            # 2^-31 of the largest weight times factor, of every value in units of its factor (|units| <= 448): `most` of it
            most = self.most(r, at, m, window, sinks, hidden)
            at += m
            tol = U[self.kind] * want.abs() * (1 + 2.0 ** -10) + (U["f16"] + 2 * off[..., None]) * weighted + 2.0 ** -25 + 2.0 ** -31 * most
            live = torch.isfinite(lse)
            held = want.to(TYPES[self.kind]).double()  # infinite where the output's type does not reach (f16: beyond 65504)
            assert torch.all(((got - want).abs() <= tol) | (got == held) & torch.isinf(held)), (r, ((got - want).abs() / tol).max().item())
            assert torch.equal(live, torch.isfinite(got_lse))
            assert torch.all((got_lse - lse)[live].abs() <= (2 * off + 2.0 ** -22 * lse.abs())[live])
            assert torch.all(got_lse[~live] == -math.inf) and torch.all(got[~live] == 0)
        assert int(self.workspace[:4096].view(torch.int32)[:256].abs().sum()) == 0  # counters are left at zero

    def most(self, r, at, m, window, sinks, hidden):
        """max over keys of weight times factor, times the sum of |values| in units, over the sum of weights: [m, heads, dim]."""
        k, v = self.held[0][r], self.held[1][r]
        n = k.shape[0]
        if n == 0 or m == 0:
            return torch.zeros(m, self.q.shape[1], self.dim, dtype=torch.float64, device="cuda")
        g = self.q.shape[1] // k.shape[1]
        t = torch.arange(n, device="cuda")
        where = self.table[r, t // self.page].long().clamp(0, self.pages - 1)
        per = self.factor[1].shape[2]
        f = torch.exp2(torch.floor(torch.log2(self.factor[1][where, :, t % self.page * per // self.page].double())))  # tokens, heads
        p = torch.arange(self.length[r] - m, self.length[r], device="cuda")[:, None]
        see = t[None] <= p
        if window:
            see &= (t[None] > p - window) | (t[None] < sinks)
        for x in (hidden or {}).get(r, ()):
            see[:, x] = False
        s = torch.einsum("nhd,thd->nht", self.q[at:at + m].double(), k.repeat_interleave(g, 1)) * self.scale
        s = s.masked_fill(~see[:, None], -math.inf)
        w = torch.exp(s - s.amax(-1, keepdim=True)).nan_to_num(0.0)
        factors = f.repeat_interleave(g, 1).T[None]
        largest = (w * factors.nan_to_num(0.0, 0.0, 0.0).clamp(min=0)).amax(-1)
        units = (v.abs() / f[..., None]).repeat_interleave(g, 1)
        total = torch.einsum("nt,thd->nhd", see.double(), units.nan_to_num(0.0, 0.0, 0.0))
        return largest[..., None] * total / w.sum(-1).clamp(min=1e-300)[..., None]


ATTEND = [
    # new, length, hq, hkv, dim, type, layout, page, block
    ([1], [1], 1, 1, 64, "bf16", "hnd", 16, 16),
    ([1, 1, 1], [5, 64, 65], 8, 2, 128, "bf16", "hnd", 16, 16),
    ([1, 1], [700, 3000], 32, 8, 128, "bf16", "nhd", 16, 16),
    ([3, 1, 0, 7], [3, 190, 40, 333], 8, 1, 128, "f16", "hnd", 32, 32),
    ([5, 2], [129, 1000], 10, 2, 64, "bf16", "nhd", 64, 32),
    ([4, 3], [128, 77], 14, 2, 256, "f16", "hnd", 64, 16),
    ([8, 8, 1], [400, 8, 1], 16, 2, 128, "bf16", "hnd", 128, 16),
    ([6, 2], [200, 515], 12, 2, 256, "bf16", "nhd", 256, 256),
    ([100, 40, 1], [100, 333, 50], 4, 2, 128, "bf16", "hnd", 16, 16),
    ([70], [200], 3, 1, 64, "f16", "hnd", 512, 64),
    ([2], [6000], 71, 1, 64, "bf16", "nhd", 1024, 128),
    ([1] * 200, [1 + 7 * i % 150 for i in range(200)], 4, 2, 64, "f16", "hnd", 16, 16),
    ([40, 30], [300, 30], 8, 2, 128, "f16", "hnd", 32, 16),
    ([8, 5], [900, 77], 16, 2, 64, "bf16", "nhd", 64, 16),
    ([4, 2], [700, 65], 16, 2, 128, "bf16", "hnd", 64, 16),
    ([0, 0, 1], [10, 0, 3], 2, 2, 64, "bf16", "hnd", 16, 16),
]


@pytest.mark.parametrize("new,length,hq,hkv,dim,kind,layout,page,block", ATTEND)
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (50, 3), (64, 70)])
def test_attend(new, length, hq, hkv, dim, kind, layout, page, block, window, sinks):
    b = Blocks(new, length, hq, hkv, dim, kind, layout, page, block, seed=len(new) + dim, exact=(window, sinks) != (64, 70))
    b.run(window, sinks)
    b.check(window, sinks)
    assert b.status.tolist() == [0] * len(new)
    first = b.out.clone()
    b.run(window, sinks)  # the same bits again: the join's order is fixed
    torch.cuda.synchronize()
    assert torch.equal(first.view(torch.int16), b.out.view(torch.int16))


@pytest.mark.parametrize("new,length,hq,hkv,dim,kind,page", [([2, 1], [400, 90], 4, 2, 128, "bf16", 16), ([6], [500], 16, 1, 128, "f16", 64),
                                                             ([3], [300], 8, 2, 64, "bf16", 32), ([2], [150], 8, 1, 256, "f16", 16)])
def test_attend_factors_far_apart(new, length, hq, hkv, dim, kind, page):
    """Factors from 2^-30 to 2^30: the product has no row of its own for each, but keeps each row's largest."""
    b = Blocks(new, length, hq, hkv, dim, kind, "hnd", page, 16, spread=30, size=1.0)
    b.run()
    b.check()


@pytest.mark.parametrize("hq,dim,kind", [(4, 128, "bf16"), (32, 128, "f16"), (8, 64, "bf16"), (4, 256, "bf16")])
def test_attend_sharp_scores(hq, dim, kind):
    """Scores of thousands, of which the largest take everything."""
    b = Blocks([3], [300], hq, 1, dim, kind, "hnd", 16, 16, size=300.0)
    b.run()
    b.check()


@pytest.mark.parametrize("hq,dim,kind", [(4, 128, "bf16"), (32, 128, "f16"), (4, 256, "f16")])
def test_attend_scores_beyond_32_bit_steps(hq, dim, kind):
    """Scores of 2^21 and more: steps of the products are wider than the scores' differences, one key takes all, and the result is
    that of some key whose score is within a step of the largest: no zeros, no NaN."""
    b = Blocks([2], [120], hq, 1, dim, kind, "hnd", 16, 16, size=1.0)
    b.scale = 2.0 ** 24
    b.run()
    torch.cuda.synchronize()
    got, lse = b.out[:2].double(), b.lse[:2].double()
    assert torch.all(torch.isfinite(got)) and torch.all(torch.isfinite(lse))
    want = ref.attend(b.q.double(), b.held[0][0], b.held[1][0], 118, b.scale)[1]
    assert torch.all((lse - want).abs() <= dim * 2.0 ** -22 * want.abs())
    assert torch.all(got.abs().amax(-1) > 0)


@pytest.mark.parametrize("kind,dim,hq", [("bf16", 128, 2), ("f16", 128, 32), ("f16", 256, 8), ("bf16", 64, 16)])
def test_attend_values_that_are_not_finite_stay_with_who_sees_them(kind, dim, hq):
    b = Blocks([4, 1], [200, 90], hq, 2, dim, kind, "hnd", 16, 16)
    for r, t in ((0, 198), (1, 5)):  # the third new token of row 0, and a token of row 1 that has left its window
        page, place = int(b.table[r, t // 16]), t % 16
        b.cache[1].view(torch.uint8)[page, place, 1, 7] = 0x7F
        if r:
            b.cache[0].view(torch.uint8)[page, place, 1, 9] = 0x7F
    b.run(window=80)
    torch.cuda.synchronize()
    expect = torch.zeros(5, hq, dim, dtype=torch.bool, device="cuda")
    expect[2:4, hq // 2:, 7] = True
    assert torch.equal(~torch.isfinite(b.out[:5].double()), expect)


def test_attend_bad_pages_and_rows():
    b = Blocks([2, 1, 1], [300, 100, 40], 8, 2, 128, "bf16", "hnd", 16, 16)
    hidden = {0: set(range(32, 48)) | set(range(160, 176)), 1: set(range(96, 100))}
    b.table[0, 2], b.table[0, 10], b.table[1, 6] = b.pages, -1, 2 ** 31 - 1
    b.run()
    b.check(hidden=hidden)
    assert b.status.tolist() == [1 << 13, 1 << 13, 0]
    b = Blocks([2, 1], [300, 20], 32, 2, 128, "f16", "hnd", 64, 32)
    b.table[0, 1] = -2 ** 31
    b.run()
    b.check(hidden={0: set(range(64, 128))})
    assert b.status.tolist() == [1 << 13, 0]
    b.status.zero_()
    b.length = [2 ** 31 - 1, 20]
    b.run()
    torch.cuda.synchronize()
    assert b.status.tolist() == [1 << 4, 0] and torch.all(b.out[:2] == 0)


def test_attend_on_another_stream_and_in_a_graph():
    b = Blocks([2, 1, 5], [500, 40, 77], 8, 2, 128, "bf16", "hnd", 16, 16)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    b.run(stream=side)
    side.synchronize()
    b.check()
    graph, lengths = torch.cuda.CUDAGraph(), _i32(b.length)
    with torch.cuda.graph(graph):
        _kv().ss_attend_blocks(b.plan, b.q, *b.cache, *b.factor, b.table, lengths, b.cu, out=b.out, row_status=b.status, workspace=b.workspace,
                               scale=b.scale, lse=b.lse)
    held = b.held
    for length in ([400, 13, 5], [500, 1, 77]):
        b.out[:8] = 7.0
        lengths.copy_(_i32(length))
        graph.replay()
        b.length, b.held = length, [[x[:n] for x, n in zip(side, length)] for side in held]
        b.check()


def test_attend_long_rows_are_split():
    """One long row over every CTA, beside rows of one token; far offsets in the factors."""
    b = Blocks([1, 2, 1], [1, 20000, 2], 4, 1, 128, "bf16", "hnd", 64, 16)
    b.run()
    torch.cuda.synchronize()
    got = b.out[1:3].double()
    q, k, v = b.q[1:3].double(), b.held[0][1][:, 0], b.held[1][1][:, 0]
    s = torch.einsum("nhd,td->nht", q, k) * b.scale
    s[0, :, 19999] = -math.inf
    w = torch.softmax(s, -1)
    want = torch.einsum("nht,td->nhd", w, v)
    tol = 2.0 ** -8 * want.abs() + 2.0 ** -10 * torch.einsum("nht,td->nhd", w, v.abs()) + 2.0 ** -20
    assert torch.all((got - want).abs() <= tol)


def test_a_step_with_the_calls_together():
    """Append, store, attention and commit over some steps, against 64 bits over what the cache holds."""
    kv = _kv()
    rows, hq, hkv, dim, page, block = 3, 8, 2, 64, 32, 16
    g = torch.Generator(device="cuda").manual_seed(5)
    pages, blocks = 24, 6
    plan = kv.Plan(max_rows=rows, max_tokens=300, max_new=4, q_heads=hq, kv_heads=hkv, head_dim=dim, page_size=page, num_pages=pages,
                   max_blocks=blocks, cache_dtype="e4m3")
    cache = [_bytes("hnd", pages, page, hkv, dim, 0x7F) for _ in range(2)]
    factor = [torch.full((pages, hkv, page // block), math.nan, device="cuda") for _ in range(2)]
    table, kv_len, seq = _i32([[-1] * blocks] * rows), _i32([0] * rows), _i32([0] * rows)
    free, count, status = torch.arange(pages, dtype=torch.int32, device="cuda"), _i32([pages]), _i32([0] * rows)
    workspace = torch.zeros(plan.workspace_bytes, dtype=torch.uint8, device="cuda")
    kept = [[], [], []]  # rounded-up bounds on what is held: the values that went in
    for step, new in enumerate(([40, 1, 90], [3, 4, 1], [4, 4, 4], [1, 2, 3])):
        n = sum(new)
        cu = _i32([0] + np.cumsum(new).tolist())
        slots, positions = _i32([0] * n), _i32([0] * n)
        q, k, v = ((torch.randn(n, h, dim, generator=g, device="cuda") * (1 + step)).to(torch.bfloat16) for h in (hq, hkv, hkv))
        out = torch.zeros(n, hq, dim, dtype=torch.bfloat16, device="cuda")
        kv.ss_kv_append(plan, table, kv_len, free, count, cu, slots=slots, positions=positions, seq_len=seq, row_status=status)
        kv.ss_kv_store_blocks(plan, k, v, *cache, *factor, table, kv_len, seq, cu, row_status=status)
        kv.ss_attend_blocks(plan, q, *cache, *factor, table, seq, cu, out=out, row_status=status, workspace=workspace, scale=0.125)
        torch.cuda.synchronize()
        assert status.tolist() == [0] * rows
        at = 0
        for r, m in enumerate(new):
            total = int(seq[r])
            t = torch.arange(total, device="cuda")
            where, place = table[r, t // page].long(), t % page
            held = [bref.decoded(c.view(torch.uint8)[where, place]) * f.double()[where, :, place // block][..., None] for c, f in zip(cache, factor)]
            kept[r] = kept[r][:total - m] + [x for x in zip(k[at:at + m].double(), v[at:at + m].double())]
            for which in range(2):  # a value is within half a step (2^-4, or a subnormal one) of what went in, twice where its block grew
                went = torch.stack([x[which] for x in kept[r]])
                top = factor[which][where, :, place // block].double()[..., None]
                assert torch.all((held[which] - went).abs() <= 2.0 ** -4 * went.abs() + 3 * 2.0 ** -10 * top)
            want, _, weighted, _, size = ref.attend(q[at:at + m].double(), *held, total - m, 0.125)
            off = dim * 2.0 ** -23 * size + 2.0 ** -20
            tol = 2.0 ** -8 * want.abs() * 1.01 + (2.0 ** -11 + 2 * off[..., None]) * weighted + 2.0 ** -20
            assert torch.all((out[at:at + m].double() - want).abs() <= tol)
            at += m
        keep = _i32([m - 1 if step % 2 and m > 1 else m for m in new])
        kv.ss_kv_commit(plan, table, kv_len, free, count, seq, counts=keep, plus=0)


def test_calls_refuse_wrong_arguments():
    from spec_verification_gb300 import native
    kv = _kv()
    b = Blocks([2], [40], 4, 2, 64, "bf16", "hnd", 32, 16)
    k = torch.zeros(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    held = _i32([38])
    cache = dict(zip(("k_cache", "v_cache", "k_scale", "v_scale"), b.cache + b.factor))
    store = dict(cache, k=k, v=k, block_table=b.table, kv_len=held, seq_len=_i32([40]), cu_new=b.cu, row_status=b.status)
    load = dict(cache, slots=_i32([0, 1]), k_out=k, v_out=k.clone())
    attend = dict(cache, q=b.q, block_table=b.table, seq_len=_i32([40]), cu_new=b.cu, out=b.out, row_status=b.status, workspace=b.workspace, scale=0.1)

    def refused(code, call, args, **change):
        with pytest.raises(native.SSError) as e:
            call(b.plan, **{**args, **change})
        assert e.value.code == code, (change.keys(), str(e.value))

    calls = [(kv.ss_kv_store_blocks, store), (kv.ss_kv_load_blocks, load), (kv.ss_attend_blocks, attend)]
    shape = b.factor[0].shape
    raw = torch.zeros(shape.numel() + 4, device="cuda")
    for call, args in calls:
        call(b.plan, **args)
        refused(-1, call, args, k_scale=b.factor[0].half())
        refused(-1, call, args, v_scale=b.factor[1][:-1])
        refused(-1, call, args, k_scale=b.factor[0][..., :1].expand(shape))
        refused(-1, call, args, k_scale=b.factor[0].flatten())
        refused(-1, call, args, v_scale=b.factor[1].cpu())
        refused(-1, call, args, k_cache=b.cache[0].view(torch.uint8))
        refused(-1, call, args, k_cache=b.cache[0][:-1])
        call(b.plan, **{**args, "k_scale": raw[1:shape.numel() + 1].view(shape)})  # any address of a float32 will do
        four = torch.ones(shape[0], 2, 4, device="cuda")  # blocks of eight tokens
        refused(-3, call, args, k_scale=four, v_scale=four)
        three = torch.ones(shape[0], 2, 3, device="cuda")
        refused(-1, call, args, k_scale=three, v_scale=three)
    refused(-1, kv.ss_kv_store_blocks, store, k=k[:1])
    refused(-1, kv.ss_kv_store_blocks, store, k=k.half())
    refused(-1, kv.ss_kv_store_blocks, store, kv_len=held.long())
    refused(-1, kv.ss_kv_store_blocks, store, B=2)
    odd = torch.zeros(2, 2 * 64 + 4, dtype=torch.bfloat16, device="cuda")[:, :128].view(2, 2, 64)
    refused(-2, kv.ss_kv_store_blocks, store, v=odd)
    refused(-2, kv.ss_kv_load_blocks, load, k_out=odd)
    refused(-1, kv.ss_kv_load_blocks, load, k_out=k[:1])
    refused(-1, kv.ss_kv_load_blocks, load, slots=_i32([0]))
    refused(-4, kv.ss_attend_blocks, attend, workspace=b.workspace[:256])
    refused(-1, kv.ss_attend_blocks, attend, scale=0.0)
    refused(-1, kv.ss_attend_blocks, attend, window=-1)
    none = torch.zeros(0, 2, 64, dtype=torch.bfloat16, device="cuda")  # no tokens: nothing is done
    kv.ss_kv_store_blocks(b.plan, **{**store, "k": none, "v": none})
    kv.ss_kv_load_blocks(b.plan, **{**load, "slots": _i32([]), "k_out": none, "v_out": none})
    wide = kv.Plan(max_rows=1, max_tokens=4, q_heads=4, kv_heads=2, head_dim=64, page_size=32, num_pages=b.pages, max_blocks=2)
    for call, args in calls:
        with pytest.raises(native.SSError):
            call(wide, **args)  # factors of blocks belong to an 8-bit cache
    torch.cuda.synchronize()
