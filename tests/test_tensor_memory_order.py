"""A kernel that lets its successor begin holds its tensor memory by then (no GPU needed: the sources are read).

The successor may allocate tensor memory before it waits for this kernel.  If it could do so on an SM where a block of this one
has not allocated yet, each would wait for the other, and neither wait has a limit."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_weight_quantized_matmul_gb300", "csrc")


def kernels():
    """(file:name, body) of every __global__ function."""
    for path in sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cuh"))):
        text = re.sub(r"//[^\n]*", "", open(path).read())
        for at in re.finditer(r"__global__\s+void", text):
            begin = text.index(") {", at.end()) + 2
            depth, end = 1, begin + 1
            while depth:
                depth += {"{": 1, "}": -1}.get(text[end], 0)
                end += 1
            name = re.search(r"(\w+_kernel)\s*\(", text[at.end():begin]).group(1)
            yield f"{os.path.basename(path)}:{name}", text[begin:end]


HOLDING = [(name, body) for name, body in kernels() if "tmem_alloc(" in body]


def test_the_kernels_are_found():
    assert {name.split(":")[1] for name, _ in HOLDING} >= {"attend_tc_kernel", "wq_tc_kernel", "wq_tcp_kernel", "wq_w4a16_kernel", "wq_w4a4_kernel"}


@pytest.mark.parametrize("name,body", HOLDING, ids=[name for name, _ in HOLDING])
def test_tensor_memory_is_allocated_before_the_successor_may_begin(name, body):
    triggers = [m.start() for m in re.finditer(r"griddep_launch_dependents\(\)", body)]
    if not triggers:
        pytest.skip("lets no successor begin before its end")
    held = body.index("__syncthreads()", body.rindex("tmem_alloc("))      # every warp has got its address
    assert min(triggers) > held
