"""CPU-side checks of the KV-cache entry points: exports and struct layouts
against include/ss_kv.h, refusals that need no device, the frequency helper."""
import ctypes as C
import math
import re
from pathlib import Path

import numpy as np
import pytest

ROOT = Path(__file__).resolve().parents[1]
HEADER = ROOT / "include" / "ss_kv.h"
ERR_ARG, ERR_UNSUPPORTED = -1, -3


@pytest.fixture(scope="module")
def kv():
    from spec_verification_gb300 import build, kv
    build.build()
    kv.library()
    return kv


def _text():
    return re.sub(r"/\*.*?\*/", "", HEADER.read_text(), flags=re.S)


def test_library_exports_every_header_function(kv):
    names = sorted(set(re.findall(r"^\s*(?:const\s+)?[A-Za-z_][A-Za-z0-9_]*\s*\**\s*(ss_[a-z0-9_]+)\s*\(", _text(), flags=re.M)))
    assert set(kv.EXPORTS) == set(names)
    for n in names:
        assert hasattr(kv.library(), n), n


def test_struct_layouts_match_header(kv):
    def fields(struct):
        body = re.search(r"typedef struct \{([^{}]*)\}\s*" + struct + ";", _text(), flags=re.S).group(1)
        out = []
        for decl in body.split(";"):
            toks = [t for t in decl.replace("*", " ").replace(",", " ").split() if t != "const"]
            out += toks[1:]
        return out

    for name, cls in [("ss_kv_config", kv.Config), ("ss_kv_cache", kv.Cache), ("ss_kv_pool", kv.Pool),
                      ("ss_rope_batch", kv.RopeBatch), ("ss_attend_batch", kv.AttendBatch)]:
        assert fields(name) == [f for f, _ in cls._fields_], name


def test_status_bits_and_types_agree(kv):
    for name, val in [("SS_ST_KV_POOL", kv.ST_KV_POOL), ("SS_ST_KV_TABLE", kv.ST_KV_TABLE), ("SS_ST_KV_PAGE", kv.ST_KV_PAGE)]:
        m = re.search(name + r" = 1u << (\d+)", _text())
        assert m and (1 << int(m.group(1))) == val, name
    assert re.search(r"SS_F16 = 2, SS_E4M3 = 3", _text()) and (kv.SS_F16, kv.SS_E4M3) == (2, 3)


GOOD = dict(max_rows=4, max_tokens=64, max_new=4, q_heads=8, kv_heads=2, head_dim=128, page_size=16, num_pages=32,
            max_blocks=8, dtype=1, cache_dtype=1, device=0)


@pytest.mark.parametrize("change,code", [
    ({"max_rows": 0}, ERR_UNSUPPORTED), ({"max_rows": 8193}, ERR_UNSUPPORTED), ({"max_tokens": 0}, ERR_UNSUPPORTED),
    ({"max_tokens": (1 << 24) + 1}, ERR_UNSUPPORTED), ({"max_new": 0}, ERR_ARG), ({"q_heads": 7}, ERR_UNSUPPORTED),
    ({"q_heads": 0}, ERR_UNSUPPORTED), ({"kv_heads": 0}, ERR_UNSUPPORTED), ({"head_dim": 96}, ERR_UNSUPPORTED),
    ({"page_size": 8}, ERR_UNSUPPORTED), ({"page_size": 48}, ERR_UNSUPPORTED), ({"page_size": 2048}, ERR_UNSUPPORTED),
    ({"num_pages": 0}, ERR_UNSUPPORTED), ({"num_pages": 1 << 27}, ERR_UNSUPPORTED), ({"max_blocks": 0}, ERR_UNSUPPORTED),
    ({"max_blocks": 1 << 27}, ERR_UNSUPPORTED), ({"dtype": 0}, ERR_ARG), ({"dtype": 3, "cache_dtype": 3}, ERR_ARG),
    ({"cache_dtype": 2}, ERR_ARG), ({"cache_dtype": 0}, ERR_ARG),
    ({"max_tokens": 1 << 24, "q_heads": 256}, ERR_UNSUPPORTED)])
def test_plan_refuses_sizes_before_any_device_query(kv, change, code):
    p = C.c_void_p(12345)
    cfg = kv.Config(**{**GOOD, **change})
    assert kv.library().ss_kv_plan_create(C.byref(p), C.byref(cfg)) == code
    assert p.value is None
    assert kv.library().ss_last_error()


def test_null_arguments_are_refused(kv):
    L = kv.library()
    cfg = kv.Config(**GOOD)
    p = C.c_void_p()
    assert L.ss_kv_plan_create(None, C.byref(cfg)) == ERR_ARG
    assert L.ss_kv_plan_create(C.byref(p), None) == ERR_ARG
    assert L.ss_kv_workspace_bytes(None) == 0
    L.ss_kv_plan_destroy(None)
    pool, rope, attend, cache = kv.Pool(), kv.RopeBatch(), kv.AttendBatch(), kv.Cache()
    assert L.ss_kv_append(None, None, None, None, None, None) == ERR_ARG
    assert L.ss_kv_append(C.byref(pool), None, None, None, None, None) == ERR_ARG
    assert L.ss_kv_commit(C.byref(pool), None, None, 0, None) == ERR_ARG
    assert L.ss_rope_store(None, None) == ERR_ARG
    assert L.ss_rope_store(C.byref(rope), C.byref(cache)) == ERR_ARG
    assert L.ss_attend(None, None) == ERR_ARG
    assert L.ss_attend(C.byref(attend), C.byref(cache)) == ERR_ARG


def test_plan_without_gpu_reports_error(kv):
    import torch
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    from spec_verification_gb300 import native
    with pytest.raises(native.SSError):
        kv.Plan(max_rows=1, max_tokens=1, q_heads=1, kv_heads=1, head_dim=64, page_size=16, num_pages=1, max_blocks=1)


@pytest.mark.parametrize("rot,base", [(64, 10000.0), (128, 500000.0), (2, 10000.0)])
def test_frequencies(kv, rot, base):
    want = [base ** (-2 * i / rot) for i in range(rot // 2)]
    np.testing.assert_allclose(kv.rope_frequencies(rot, base), want, rtol=1e-14)
    np.testing.assert_allclose(kv.rope_frequencies(rot, base, factor=4.0), np.array(want) / 4, rtol=1e-14)


def test_frequencies_blended_for_long_contexts(kv):
    rot, base, factor, length, low, high = 128, 10000.0, 8.0, 4096, 1.0, 32.0
    got = kv.rope_frequencies(rot, base, factor=factor, original_len=length, low_turns=low, high_turns=high)
    seen = set()
    for i in range(rot // 2):
        f = base ** (-2 * i / rot)
        turns = length * f / (2 * math.pi)
        if turns >= high:
            want, kind = f, "kept"
        elif turns <= low:
            want, kind = f / factor, "stretched"
        else:
            stay = (turns - low) / (high - low)
            want, kind = f * stay + f / factor * (1 - stay), "blended"
        seen.add(kind)
        assert got[i] == pytest.approx(want, rel=1e-13)
    assert seen == {"kept", "stretched", "blended"}


def test_frequencies_refusals(kv):
    from spec_verification_gb300 import native
    for kw in [dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=64, base=0.0), dict(rot_dim=64, base=math.inf),
               dict(rot_dim=64, factor=0.5), dict(rot_dim=64, factor=math.nan), dict(rot_dim=64, original_len=-1),
               dict(rot_dim=64, original_len=10, low_turns=2.0, high_turns=2.0)]:
        with pytest.raises(native.SSError):
            kv.rope_frequencies(**kw)
