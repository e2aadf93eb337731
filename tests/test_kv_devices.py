"""The KV-cache calls refuse tensors of another device than their plan's, whose addresses mean nothing to its kernels.
On the CPU: host tensors that say they are on one device or another; a refusal comes before the library is called."""
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")


class On:
    """A tensor that says it is on cuda:n."""

    def __init__(self, tensor, n):
        self.__dict__.update(tensor=tensor, n=n)

    def __getattr__(self, name):
        return getattr(self.tensor, name)

    is_cuda = True
    device = property(lambda self: torch.device("cuda", self.n))

    def get_device(self):
        return self.n

    def __getitem__(self, i):
        return On(self.tensor[i], self.n)


def _i32(n):
    return torch.zeros(n, dtype=torch.int32)


def _calls(kv):
    plan = SimpleNamespace(device=1, handle=0, q_heads=4, kv_heads=2, head_dim=64, max_blocks=3, num_pages=5, page_size=16,
                           type=torch.bfloat16, cache_type=torch.float8_e4m3fn, cache_shape=torch.Size((5, 16, 2, 64)))
    bf16 = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16)  # noqa: E731
    cache = dict(k_cache=torch.zeros(5, 16, 2, 64).to(torch.float8_e4m3fn), v_cache=torch.zeros(5, 16, 2, 64).to(torch.float8_e4m3fn),
                 k_scale=torch.ones(2), v_scale=torch.ones(2))
    pool = dict(block_table=_i32(6).view(2, 3), kv_len=_i32(2), free_pages=_i32(5), free_count=_i32(1), seq_len=_i32(2))
    attend = dict(cache, q=bf16(4, 4, 64), block_table=_i32(6).view(2, 3), seq_len=_i32(2), cu_new=_i32(3), out=bf16(4, 4, 64), row_status=_i32(2),
                  workspace=torch.zeros(256, dtype=torch.uint8), lse=torch.zeros(4, 4))
    rope = dict(cache, q=bf16(4, 4, 64), k=bf16(4, 2, 64), v=bf16(4, 2, 64), inv_freq=torch.ones(32, dtype=torch.float64), positions=_i32(4),
                slots=_i32(4), q_out=bf16(4, 4, 64), q_weight=bf16(64), k_weight=bf16(64))
    return plan, [(kv.ss_kv_append, dict(pool, cu_new=_i32(3), slots=_i32(4), positions=_i32(4), row_status=_i32(2)), {}),
                  (kv.ss_kv_commit, dict(pool, counts=_i32(2), finished=_i32(2)), {}),
                  (kv.ss_rope_store, rope, {}), (kv.ss_attend, attend, {"scale": 0.125})]


def test_tensors_of_another_device_are_refused():
    from spec_verification_gb300 import build, kv, native
    build.build()
    kv.library()
    plan, calls = _calls(kv)
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


@pytest.mark.parametrize("workspace", [torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros(1 << 12, dtype=torch.uint8)[::2],
                                       torch.zeros(4, 256, dtype=torch.uint8).T], ids=["expanded", "strided", "turned"])
def test_workspaces_that_are_not_contiguous_are_refused(workspace):
    """Their number of elements does not say how many bytes are there from their address on."""
    from spec_verification_gb300 import build, kv, native
    build.build()
    kv.library()
    plan, calls = _calls(kv)
    _, tensors, others = calls[-1]
    args = {n: On(t, 1) for n, t in {**tensors, "workspace": workspace}.items()}
    with pytest.raises(native.SSError) as e:
        kv.ss_attend(plan, **args, **others, stream=SimpleNamespace(cuda_stream=0))
    assert e.value.code == -1 and "contiguous" in str(e.value)
