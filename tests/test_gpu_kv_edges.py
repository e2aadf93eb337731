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
