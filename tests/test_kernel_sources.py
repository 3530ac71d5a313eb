"""Orders in the kernels' sources that no run can show without hanging."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "combine_device_resident_gb300", "csrc")


def kernels():
    for name in sorted(os.listdir(CSRC)):
        if name.endswith(".cu"):
            for body in open(os.path.join(CSRC, name)).read().split("__global__")[1:]:
                yield name, re.search(r"(\w+_kernel)\(", body).group(1), body


def test_tensor_memory_is_taken_after_the_dependency_wait():
    """A kernel that starts early and takes tensor memory before it waits can leave its predecessor, whose blocks may
    take theirs later, without any: each would wait for the other."""
    found = set()
    for name, kernel, body in kernels():
        alloc = min((body.find(t) for t in ("tcgen05.alloc", "tmem_alloc_all(") if t in body), default=-1)
        if alloc >= 0:
            found.add(kernel)
            assert 0 <= body.find("grid_dependency_wait();") < alloc, (name, kernel)
    assert found >= {"expert_gemm_kernel", "expert_w4_tmem_kernel"}


def test_tensor_memory_loads_are_used_after_their_wait():
    """The registers of an asynchronous load are no operands of the wait, so a compiler may use them before it, unless they
    pass through a statement behind it, in the same function."""
    found = 0
    for name in sorted(os.listdir(CSRC)):
        text = open(os.path.join(CSRC, name)).read()
        for wait in re.finditer(r"tcgen05\.wait::ld", text):
            found += 1
            assert re.search(r'asm volatile\("" : "\+[fr]"', text[wait.end():text.index("\n}", wait.end())]), name
    assert found
