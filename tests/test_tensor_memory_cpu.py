"""Every kernel takes its tensor memory after its wait for the previous kernel and before
the next one may start, held on the source text: a previous kernel that lets this one
start before its own allocation would wait for these columns, and this kernel for its
end; no healthy run shows it."""
import os
import re

import pytest

from gated_delta_rule_150_b200 import build as gdr_build


def _kernels():
    for path in gdr_build.sources():
        with open(path) as f:
            src = re.sub(r"//[^\n]*", "", f.read())
        for body in src.split("__global__")[1:]:
            if re.search(r"\btmem_alloc(_pair)?\(", body):
                yield pytest.param(body, id=os.path.basename(path) + ":" + re.search(r"(\w+_kernel)\(", body).group(1))


KERNELS = list(_kernels())


def test_the_kernels_are_found():
    assert len(KERNELS) == 4


@pytest.mark.parametrize("body", KERNELS)
def test_order(body):
    first = lambda p: min((m.start() for m in re.finditer(p, body)), default=-1)
    wait, alloc, start = first(r"\bpdl_wait\(\)"), first(r"\btmem_alloc(_pair)?\("), first(r"\bpdl_launch_dependents\(\)")
    assert 0 <= wait < alloc < start
