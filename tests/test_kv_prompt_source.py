"""Static checks of the prompt kernel's source: what is shown by reading, as it needs warps that lag behind one another."""
import re

from tests.test_kv_source import _body, _code


def test_a_place_in_the_ring_is_not_brought_anew_before_the_guard_has_passed_it():
    """The guard follows the ring by parities, which tell a phase from the next only: so whoever gives a slot of values back
    has waited for the guard, in every tile and not only in those that it has to look at."""
    code = _code("ss_kv_prompt.cuh")
    values = _body(code, code.index("__device__ void values_warp("))
    guard = _body(code, code.index("__device__ void guard_warps("))
    release = values.index("commit(&c.empty[")
    look = values.index("done(&c.ready[number % kMaxSlots]")
    wait = re.search(r"if \(!__all_sync\(0xffffffffu, looked\)\) w\.wait\(&c\.ready\[number % kMaxSlots\]", values)
    assert look < wait.start() < release
    for at in (look, wait.start()):  # neither inside a block of cut tiles alone
        for m in re.finditer(r"if \(cut[^)]*\) \{", values):
            assert not m.end() < at < m.end() + len(_body(values, m.end() - 1))
    assert "arrive(&c.ready[nth % kMaxSlots])" in guard
    for m in re.finditer(r"if \(cut\) \{", guard):
        assert "arrive(&c.ready" not in _body(guard, m.end() - 1)


def test_waits_of_the_softmax_follow_from_the_unit_alone():
    """No barrier brings warps together between the start of the kernel and its end: a warp whose wait ran out leaves without
    the others."""
    code = _code("ss_kv_prompt.cuh")
    softmax = _body(code, code.index("__device__ void softmax_warps("))
    assert "bar.sync" not in softmax and "__syncthreads" not in softmax and not re.search(r"\bbar_", softmax)
