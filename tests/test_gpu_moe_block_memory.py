"""The example block makes its buffers once."""
import pytest
import torch

from tests.test_gpu_moe_block import make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("form", ["bf16", "8bit", "4bit"])
def test_a_call_allocates_nothing(form):
    b, x, r = make(form)
    first = b(x, r.clone()).clone()  # (the first product of a process makes the library's workspace)
    residual = r.clone()
    torch.cuda.synchronize()
    before = torch.cuda.memory_stats()["allocation.all.allocated"]
    out = b(x, residual)
    assert torch.cuda.memory_stats()["allocation.all.allocated"] == before
    assert torch.equal(out, first)
    b.close()
