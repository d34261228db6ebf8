"""Orders in the linear-attention kernels' sources on which their launches' progress rests, read from the text: a
wrong order would show on a GPU as a hang only, so it is never run."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "delta_rule_linear_gb300", "csrc")


def _kernels():
    for path in sorted(glob.glob(os.path.join(CSRC, "linear_*.cu"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        parts = re.split(r"__global__ void", text)[1:]
        for body in parts:
            name = re.search(r"(linear_\w+_kernel)\s*\(", body)
            if name:
                yield name.group(1), body


def test_sources_are_read():
    names = [n for n, _ in _kernels()]
    assert {"linear_state_kernel", "linear_local_kernel", "linear_grad_kernel", "linear_chunk_kernel"} <= set(names)


@pytest.mark.parametrize("name,body", [(n, b) for n, b in _kernels() if "tmem_alloc(" in b], ids=lambda x: x if len(x) < 60 else "")
def test_the_next_launch_may_start_only_after_the_tmem_allocation(name, body):
    """A CTA of the next launch takes all TMEM of an SM and then waits for this one: this one has to have its own by
    then, which a barrier after the allocation makes sure of."""
    if "next_may_start(" not in body:
        return
    alloc = body.index("tmem_alloc(")
    barrier = body.index("__syncthreads()", alloc)
    assert body.index("next_may_start(") > barrier, name
