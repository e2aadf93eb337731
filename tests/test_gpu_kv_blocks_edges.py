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
