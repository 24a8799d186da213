"""Rules of the 8-bit product's kernels that no run on a healthy GPU shows, held on
the source text (linear_fp8.cu): where they break, a kernel that gives up a wait
would release memory that is still written, or two kernels would wait for each other."""
import os
import re

import pytest

from gated_delta_rule_150_b200 import build as gdr_build


def _source():
    with open(os.path.join(gdr_build.CSRC, "linear_fp8.cu")) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _enclosing_ifs(src, at):
    """Conditions of the `if`s around position `at`: of each open block, and of the
    statement itself."""
    conds, depth = [], 0
    start = max(src.rfind(c, 0, at) for c in ";{}")
    conds += re.findall(r"if \((.*)\)\s*$", src[start + 1:at].strip() + "\n", re.M)
    for i in range(at - 1, -1, -1):
        if src[i] == "}":
            depth += 1
        elif src[i] == "{":
            if depth:
                depth -= 1
            else:
                head = src[max(src.rfind(c, 0, i) for c in ";{}") + 1:i]
                conds += re.findall(r"if \((.*)\)\s*$", head.strip() + "\n", re.M | re.S)
    return conds


@pytest.mark.parametrize("call", ["mma_e4m3(", "mma_e4m3_pair(", "mma_commit(", "mma_commit_pair("])
def test_mmas_and_their_commits_are_issued_by_the_elected_lane(call):
    """A commit follows the MMAs of the thread that issues it, and no other's."""
    src = _source()
    places = [m.start() for m in re.finditer(r"(?<![\w])" + re.escape(call), src)]
    assert places
    for at in places:
        assert any("elect_one()" in c for c in _enclosing_ifs(src, at)), src[at - 80:at + 40]


@pytest.mark.parametrize("kernel", ["linear_few_kernel", "linear_pair_kernel"])
def test_tensor_memory_is_held_only_after_the_previous_kernel(kernel):
    """A kernel that the next one may overlap could let it start before its own
    allocation: were tensor memory taken before the wait for that kernel's end, each
    would wait for the other.  For the same reason the kernel after this one may start
    only once this one has its columns."""
    src = _source()
    body = src[src.index(kernel + "("):]
    body = body[:body.index("__global__") if "__global__" in body else len(body)]
    places = [[m.start() for m in re.finditer(p, body)]
              for p in (r"\bpdl_wait\(\)", r"\btmem_alloc(_pair)?\(", r"\bpdl_launch_dependents\(\)")]
    assert [len(p) for p in places] == [1, 1, 1]
    wait, alloc, start = (p[0] for p in places)
    assert wait < alloc < start
    alloc_ifs, start_ifs = _enclosing_ifs(body, alloc), _enclosing_ifs(body, start)
    assert alloc_ifs and alloc_ifs == start_ifs           # by the allocating warp, after it
