"""The norm and the experts' products on inputs at the ends of their ranges:
outliers, far gates, infinities, the smallest rows; each against 64 bits, with
the tolerances that `tests/test_gpu_experts.py` derives.
"""
import numpy as np
import pytest
import torch

import combine_device_resident_gb300 as A
from tests.test_gpu_experts import BF, CANARY, DEV, gen, layout, normal, plan_for, product_ref, within

pytestmark = pytest.mark.gpu

# expert rows of the 4-bit products below, and output widths that take either of their forms
ROWS4 = [[5, 40, 0, 20]]
WIDTHS4 = {"split": 72, "tensor memory": 3600}


def w4_call(x, w4, ws, N, group):
    """y of one 4-bit call on rows x [65][K], and (expert, first row, end) of each expert."""
    plan = plan_for(np.array(ROWS4))
    sp, segs = layout(plan, np.array(ROWS4))
    y = torch.full((x.shape[0], N), CANARY, device=DEV, dtype=torch.bfloat16)
    plan.expert_matmul_w4(x, w4, ws, sp, y)
    torch.cuda.synchronize()
    assert plan.read_status() == 0
    plan.close()
    return y, segs


# ---- 4-bit weights: rows with outliers -------------------------------------------------

@pytest.mark.parametrize("outlier", [1e3, 1e4, 1e5, 1e8])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N", list(WIDTHS4.values()), ids=list(WIDTHS4))
def test_w4_outliers_on_weights_of_zero(N, group, outlier):
    """A weight of zero takes its activation out of the sum, however large: the bound is in sum |x * w|."""
    K, g = 512, gen(group)
    x, w = normal(g, 65, K), normal(g, 4, N, K) * K ** -0.5
    for k in (3, 64, 65, 300):
        x[:, k] = outlier * torch.sign(x[:, k])
        w[..., k] = 0.0
    x = x.bfloat16()
    w4, ws = A.pack_weights_w4(w, group)
    w64 = A.unpack_weights_w4(w4, ws).double()
    assert (w64[..., 300] == 0).all()
    y, segs = w4_call(x, w4, ws, N, group)
    for e, a, b in segs:
        within(y[a:b], *product_ref("int4", x[a:b].double(), w64[e], ws, False, K))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N", list(WIDTHS4.values()), ids=list(WIDTHS4))
def test_w4_rows_far_from_zero(N, group):
    """Rows with a mean: the products cancel in the sum, no more than their magnitudes allow."""
    K, g = 512, gen(group)
    x = (normal(g, 65, K) + 200.0).bfloat16()
    w4, ws = A.pack_weights_w4(normal(g, 4, N, K) * K ** -0.5, group)
    w64 = A.unpack_weights_w4(w4, ws).double()
    y, segs = w4_call(x, w4, ws, N, group)
    for e, a, b in segs:
        within(y[a:b], *product_ref("int4", x[a:b].double(), w64[e], ws, False, K))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N", list(WIDTHS4.values()), ids=list(WIDTHS4))
def test_w4_large_finite_rows(N, group):
    """(q - 8) * x within fp32: the result is finite and right."""
    K, g = 256, gen(group)
    x = normal(g, 65, K)
    x[:, 100] = 2e37  # eight times it is the largest product
    x = x.bfloat16()
    w4, ws = A.pack_weights_w4(normal(g, 4, N, K) * K ** -0.5, group)
    w64 = A.unpack_weights_w4(w4, ws).double()
    y, segs = w4_call(x, w4, ws, N, group)
    for e, a, b in segs:
        within(y[a:b], *product_ref("int4", x[a:b].double(), w64[e], ws, False, K))


@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("N", list(WIDTHS4.values()), ids=list(WIDTHS4))
def test_w4_infinite_rows(N, group):
    """An infinity gives infinities of the weights' signs, and NaN on weights of zero, as in the formula."""
    K, g = 256, gen(group)
    x = normal(g, 65, K)
    x[2, 100], x[30, 5] = float("inf"), float("-inf")
    x = x.bfloat16()
    w4, ws = A.pack_weights_w4(normal(g, 4, N, K) * K ** -0.5, group)
    w64 = A.unpack_weights_w4(w4, ws).double()
    y, segs = w4_call(x, w4, ws, N, group)
    for row, k, sign, e in ((2, 100, 1.0, 0), (30, 5, -1.0, 1)):
        w = w64[e][:, k]
        assert torch.equal(torch.isnan(y[row]), w == 0)
        assert torch.equal(y[row][w != 0].double(), torch.sign(w[w != 0]) * sign * float("inf"))
    for e, a, b in segs:
        rows = [r for r in range(a, b) if r not in (2, 30)]
        within(y[rows], *product_ref("int4", x[rows].double(), w64[e], ws, False, K))
