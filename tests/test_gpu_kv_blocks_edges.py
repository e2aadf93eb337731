"""The 8-bit cache with factors of blocks at the ends of types and counts (bounds as in tests/test_gpu_kv_blocks.py: bit for bit)."""
import math

import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_kv_blocks import Store, _i32, _kv  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _env():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    from spec_verification_gb300 import build
    build.build()


def test_large_f16_values_come_back_finite():
    """From 63488 on a value is held as 256 * 2^8 = 65536, which f16 does not have: what comes back is the largest that it has."""
    s = Store(1, 32, 2, 64, "f16", "hnd", 16, 16)
    x = torch.zeros(20, 2, 64, dtype=torch.float16, device="cuda")
    x[0, 0, :8] = torch.tensor([63456.0, 63488.0, 65504.0, -63456.0, -63488.0, -65504.0, math.nan, 61440.0])
    x[17, 1, :4] = torch.tensor([math.inf, -math.inf, 57344.0, math.nan])
    s.call(x, -x, [0], [20])
    s.expect(x, -x, [0], [20])
    s.check()
    slots = [int(s.table[0, t // 16]) * 16 + t % 16 for t in range(20)]
    k_out, v_out = torch.empty_like(x), torch.empty_like(x)
    _kv().ss_kv_load_blocks(s.plan, *s.cache, *s.factor, _i32(slots), k_out=k_out, v_out=v_out)
    torch.cuda.synchronize()
    want = torch.zeros_like(x)
    want[0, 0, :8] = torch.tensor([61440.0, 65504.0, 65504.0, -61440.0, -65504.0, -65504.0, math.nan, 61440.0])
    want[17, 1, :4] = torch.tensor([57344.0, -57344.0, 57344.0, math.nan])  # infinities are held as 448 * 2^7 = 57344
    for out, sign in ((k_out, 1.0), (v_out, -1.0)):
        assert torch.equal(out.isnan(), want.isnan())
        assert torch.equal(out.nan_to_num(0.0), (sign * want).nan_to_num(0.0))
    # factors that a user wrote
    for factor, bits in ((2.0 ** 40, 0x7E), (2.0 ** 9, 0x70), (2.0 ** 9, 0x6F)):
        for c, f in zip(s.cache, s.factor):
            c.view(torch.uint8).fill_(bits)
            f.fill_(factor)
        _kv().ss_kv_load_blocks(s.plan, *s.cache, *s.factor, _i32(slots), k_out=k_out, v_out=v_out)
        torch.cuda.synchronize()
        held = (8 + (bits & 7)) * 2.0 ** ((bits >> 3) - 10) * factor
        assert torch.all(k_out == min(held, 65504.0)) and torch.all(v_out == min(held, 65504.0))


def test_more_runs_than_32_bits_count():
    """Prefix sums that go up and down: 2050 rows of 2^24 tokens each, on pages that are none, in 2^20 blocks each, between two rows of
    16 tokens on pages that are some."""
    rises, n = 2050, 1 << 24
    rows, blocks = 2 * rises + 3, n // 1024
    plan = _kv().Plan(max_rows=rows, max_tokens=n, q_heads=1, kv_heads=1, head_dim=64, page_size=1024, num_pages=2, max_blocks=blocks,
                      dtype="bf16", cache_dtype="e4m3")
    x = torch.zeros(n, 1, 64, dtype=torch.bfloat16, device="cuda")
    x[:16] = 3.5
    cache = torch.zeros(2, 2, 1024, 1, 64, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    factor = torch.full((2, 2, 1, 64), 7.0, device="cuda")
    table = torch.full((rows, blocks), -1, dtype=torch.int32, device="cuda")
    table[0, 0], table[-1, 0] = 1, 0
    held, status = _i32([0] * rows), _i32([0] * rows)
    seq, cu = _i32([16, 0] + [n, 0] * rises + [16]), _i32([0, 16] + [0, n] * rises + [0, 16])
    _kv().ss_kv_store_blocks(plan, x, -x, *cache, *factor, table, held, seq, cu, row_status=status)
    torch.cuda.synchronize()
    assert status.tolist() == [0, 1 << 9] + [1 << 13, 1 << 9] * rises + [0]
    for c, f, sign in zip(cache, factor, (1.0, -1.0)):  # 3.5 = 448 * 2^-7
        assert torch.all(c.float()[:, :16] == sign * 448.0) and torch.all(c.float()[:, 16:] == 0)
        assert torch.all(f[:, 0, 0] == 2.0 ** -7) and torch.all(f[:, 0, 1:] == 7.0)
