"""Static checks of the attention kernels' sources: what is shown by reading, as it needs a wait that runs out."""
import re
from pathlib import Path

CSRC = Path(__file__).resolve().parents[1] / "spec_verification_gb300" / "csrc"


def _code(name):
    return re.sub(r"//[^\n]*", "", (CSRC / name).read_text())


def _body(code, start):
    """The braces' contents after `start`."""
    at = code.index("{", start)
    depth = 0
    for i in range(at, len(code)):
        depth += {"{": 1, "}": -1}.get(code[i], 0)
        if depth == 0:
            return code[at + 1:i]
    raise AssertionError("unbalanced braces")


def test_softmax_warps_meet_whatever_one_of_them_has_read():
    """A warp whose wait ran out goes on with words that the others may read differently: whether it meets the others at
    the barrier inside a tile must follow from the segment alone, which all have read behind a barrier."""
    code = _code("ss_kv_attend.cuh")
    softmax = _body(code, code.index("__device__ void softmax_warps("))
    meets = [m.start() for m in re.finditer(r"any_softmax\(", softmax)]
    assert len(meets) == 2  # a segment's start, and inside a tile
    guards = [m for m in re.finditer(r"if \((\w+)\) \{", softmax) if m.end() < meets[1] < m.start() + len(m.group(0)) + len(_body(softmax, m.start()))]
    assert [g.group(1) for g in guards] == ["cut"]
    assert re.search(r"const bool cut = partly\(P, g\.u, base\)", softmax)
    assert re.search(r"const int base = tile_of\(g\.u, g\.from \+ i\) \* kTile;", softmax)
    partly = code[code.index("bool partly("):]
    assert partly.startswith("bool partly(const AttendParams& P, const Unit& u, int base)")
    assert set(re.findall(r"\b[a-zA-Z]\w*", _body(partly, 0))) <= {"return", "base", "kTile", "u", "pos0", "pos1", "P", "window", "sinks"}


def test_queries_that_may_be_overwritten_are_not_read_as_read_only():
    """ss_rope_store allows q_out to be q; a read-only load is defined only for what the kernel does not write."""
    code = _code("ss_kv_rope.cu")
    load = _body(code, code.index("auto load = [&]"))
    assert "P.q" in load and "__ldg" not in load
    uses = [m.start() for m in re.finditer(r"__ldg\(", code)]
    assert [re.search(r"__ldg\(reinterpret_cast<const uint4\*>\(v \+", code[at:at + 60]) is not None for at in uses] == [True]
    assert "__restrict__" not in code
