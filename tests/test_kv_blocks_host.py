"""CPU-side checks of the calls on an 8-bit cache with a factor for each block, and of the attention over prompts: struct layouts against include/ss_kv.h,
refusals that need no device, tensors of another device than their plan's."""
import ctypes as C
import re
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")

from tests.test_kv_devices import On, _i32  # noqa: E402
from tests.test_kv_host import ERR_ARG, _text  # noqa: E402


@pytest.fixture(scope="module")
def kv():
    from spec_verification_gb300 import build, kv
    build.build()
    kv.library()
    return kv


def test_struct_layouts_match_header(kv):
    def fields(struct):
        body = re.search(r"typedef struct \{([^{}]*)\}\s*" + struct + ";", _text(), flags=re.S).group(1)
        out = []
        for decl in body.split(";"):
            toks = [t for t in decl.replace("*", " ").replace(",", " ").split() if t != "const"]
            out += toks[1:]
        return out

    for name, cls in [("ss_kv_block_cache", kv.BlockCache), ("ss_store_batch", kv.StoreBatch), ("ss_load_batch", kv.LoadBatch),
                      ("ss_prompt_batch", kv.PromptBatch)]:
        assert fields(name) == [f for f, _ in cls._fields_], name


def test_null_arguments_are_refused(kv):
    L = kv.library()
    cache, attend, store, load = kv.BlockCache(), kv.AttendBatch(), kv.StoreBatch(), kv.LoadBatch()
    for call, batch in ((L.ss_kv_store_blocks, store), (L.ss_kv_load_blocks, load), (L.ss_attend_blocks, attend)):
        assert call(None, None) == ERR_ARG
        assert call(C.byref(batch), None) == ERR_ARG
        assert call(C.byref(batch), C.byref(cache)) == ERR_ARG
        assert call(None, C.byref(cache)) == ERR_ARG
    prompt = kv.PromptBatch()
    assert L.ss_attend_prompt(None) == ERR_ARG
    assert L.ss_attend_prompt(C.byref(prompt)) == ERR_ARG


def test_tensors_of_another_device_are_refused(kv):
    from spec_verification_gb300 import native
    plan = SimpleNamespace(device=1, handle=0, q_heads=4, kv_heads=2, head_dim=64, max_blocks=3, num_pages=5, page_size=32, cache_dtype="e4m3",
                           type=torch.bfloat16, cache_type=torch.float8_e4m3fn, cache_shape=torch.Size((5, 32, 2, 64)))
    bf16 = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16)  # noqa: E731
    cache = dict(k_cache=torch.zeros(5, 32, 2, 64).to(torch.float8_e4m3fn), v_cache=torch.zeros(5, 32, 2, 64).to(torch.float8_e4m3fn),
                 k_scale=torch.ones(5, 2, 2), v_scale=torch.ones(5, 2, 2))
    rows = dict(block_table=_i32(6).view(2, 3), seq_len=_i32(2), cu_new=_i32(3), row_status=_i32(2))
    calls = [(kv.ss_kv_store_blocks, dict(cache, **rows, k=bf16(4, 2, 64), v=bf16(4, 2, 64), kv_len=_i32(2)), {}),
             (kv.ss_kv_load_blocks, dict(cache, slots=_i32(4), k_out=bf16(4, 2, 64), v_out=bf16(4, 2, 64)), {}),
             (kv.ss_attend_blocks, dict(cache, **rows, q=bf16(4, 4, 64), out=bf16(4, 4, 64), lse=torch.zeros(4, 4),
                                        workspace=torch.zeros(256, dtype=torch.uint8)), {"scale": 0.125}),
             (kv.ss_attend_prompt, dict(q=bf16(4, 4, 64), k=bf16(4, 2, 64), v=bf16(4, 2, 64), cu_seq=_i32(3), out=bf16(4, 4, 64), row_status=_i32(2),
                                        lse=torch.zeros(4, 4), workspace=torch.zeros(256, dtype=torch.uint8)), {"scale": 0.125})]
    stream = SimpleNamespace(cuda_stream=0)
    for call, tensors, others in calls:
        for name in tensors:
            args = {n: On(t, 0 if n == name else 1) for n, t in tensors.items()}
            with pytest.raises(native.SSError) as e:
                call(plan, **args, **others, stream=stream)
            assert e.value.code == -1 and "cuda:0" in str(e.value) and "cuda:1" in str(e.value), (call.__name__, name, str(e.value))
            args[name] = tensors[name]
            with pytest.raises(native.SSError) as e:
                call(plan, **args, **others, stream=stream)
            assert e.value.code == -1 and "host" in str(e.value), (call.__name__, name, str(e.value))
        if call is kv.ss_attend_prompt:
            continue
        with pytest.raises(native.SSError) as e:  # a plan with a 16-bit cache
            call(SimpleNamespace(**{**plan.__dict__, "cache_dtype": "bf16"}), **{n: On(t, 1) for n, t in tensors.items()}, **others, stream=stream)
        assert e.value.code == -1 and "e4m3" in str(e.value)
