"""The norm and the experts' products on inputs at the ends of their ranges:
outliers, far gates, infinities, the smallest rows; each against 64 bits, with
the tolerances that `tests/test_gpu_experts.py` derives.
"""
import numpy as np
import pytest
import torch

import combine_device_resident_gb300 as A
from tests.test_gpu_experts import (BF, CANARY, DEV, check_rows8, gen, layout, norm_ref, normal, plan_for, product_ref,
                                    run_product, within)

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


# ---- the activation far out ------------------------------------------------------------

FORMS = [("bf16", 8), ("e4m3", 8), ("int4", 8), ("int4", 3600)]  # 4-bit weights: either form, by the width


def gated(kind, N, gates, up):
    """y [len(gates)][N] of one expert whose gate is gates[r] in row r and whose up is `up`, both exact."""
    n, K = len(gates), 64
    plan = A.Plan(1, 1, n, 64, 1, device=DEV, recv_order="expert")
    sp, _ = layout(plan, np.array([[n]]))
    x = torch.zeros(n, K, device=DEV)
    x[:, 0], x[:, 1] = torch.tensor(gates, device=DEV), up
    w = torch.zeros(1, 2 * N, K, device=DEV)
    w[0, :N, 0], w[0, N:, 1] = 1.0, 1.0
    y = torch.full((n, N), CANARY, device=DEV, dtype=torch.bfloat16)
    if kind == "bf16":
        plan.expert_matmul(x.bfloat16(), w.bfloat16(), sp, y, activation="swiglu")
    elif kind == "e4m3":  # a scale of 8 for the row holds a gate and an up of up to 3584 in steps of theirs
        rows8 = plan.new_rows8(n, K)
        q, s = A.rows8_parts(rows8)
        s.fill_(8.0)
        q.copy_((x / 8.0).to(torch.float8_e4m3fn))
        assert torch.equal(q.float() * 8.0, x)
        plan.expert_matmul(rows8, w.to(torch.float8_e4m3fn), sp, y, w_scale=torch.ones(1, 2 * N, device=DEV),
                           activation="swiglu")
    else:
        words = torch.zeros(1, 2 * N, K // 8, dtype=torch.int32, device=DEV)
        words[...] = -0x77777778  # eight eights: weights of zero
        words[0, :N, 0] += 1        # k = 0: 9 - 8
        words[0, N:, 0] += 1 << 16  # k = 1
        assert torch.equal(A.unpack_weights_w4(words, torch.ones(1, 2 * N, 1, device=DEV)), w)
        plan.expert_matmul_w4(x.bfloat16(), words, torch.ones(1, 2 * N, 1, device=DEV, dtype=torch.bfloat16), sp, y,
                              activation="swiglu")
    torch.cuda.synchronize()
    assert plan.read_status() == 0
    plan.close()
    return y


@pytest.mark.parametrize("kind,N", FORMS)
def test_gates_far_out(kind, N):
    """silu is g exp(g) there, down to where bf16 ends: fp32's exp and division are (8 + 2|g|) * 2^-23 off, half a step
    of a bf16 below its smallest normal is 2^-134, and below fp32's the power is a step of 2^-149 off, times g and the
    up."""
    gates = [-72.0, -80.0, -88.0, -96.0, -104.0, 72.0, 88.0, 96.0, 104.0, 2048.0, -2048.0, 8.0, -8.0, 0.0]
    y = gated(kind, N, gates, 64.0).double()
    g = torch.tensor(gates, device=DEV, dtype=torch.float64)
    ref = (g / (1.0 + torch.exp(-g)) * 64.0).unsqueeze(-1).expand_as(y)
    rel = (BF + (8 + 2 * g.abs()) * 2.0 ** -23).unsqueeze(-1)
    within(y, ref, ref.abs() * rel + 2.0 ** -134 + ((g.abs() + 2) * 64 * 2.0 ** -149).unsqueeze(-1))


@pytest.mark.parametrize("kind,N", [f for f in FORMS if f[0] != "e4m3"])  # 8-bit rows hold no such pair exactly
def test_overflowing_sums_stay_infinite(kind, N):
    """A product past fp32 is an infinity of its sign, not a NaN (gate 2048, up 2^126)."""
    big = 2.0 ** 126
    y = gated(kind, N, [2048.0, -2048.0, 8.0, -1.0], big).double()
    assert (y[0] == float("inf")).all() and (y[1] == 0).all() and (y[2] == float("inf")).all()
    ref = torch.full((N,), -1.0 / (1.0 + np.exp(1.0)) * big, dtype=torch.float64, device=DEV)
    within(y[3], ref, ref.abs() * (BF + 10 * 2.0 ** -23))


@pytest.mark.parametrize("kind,N", FORMS)
def test_a_large_gate_is_the_gate(kind, N):
    y = gated(kind, N, [704.0, 960.0, 112.0, -112.0], 8.0).double()
    for row, want in ((0, 704.0 * 8), (1, 960.0 * 8), (2, 112.0 * 8)):
        within(y[row], torch.full_like(y[row], want), torch.full_like(y[row], want * (BF + 2.0 ** -20)))
    assert (y[3].abs() < 1e-37).all()


# ---- refusals --------------------------------------------------------------------------

@pytest.mark.parametrize("kind", ["e4m3", "int4"])
@pytest.mark.parametrize("at", ["first", "last"])
def test_output_over_the_weights_scales_is_refused(kind, at):
    """The scales are read while other blocks store y."""
    plan = A.Plan(1, 2, 16, 64, 1, device=DEV, recv_order="expert")
    sp, _ = layout(plan, np.array([[9, 7]]))
    K, N, rows = 64, 32, plan.arena_rows
    size = 2 * N * (4 if kind == "e4m3" else K // 32 * 2)
    buf = torch.zeros(size + rows * N * 2, dtype=torch.uint8, device=DEV)
    # y covers the first or the last 16 bytes of the scales
    y0 = buf.numel() - rows * N * 2 if at == "last" else 0
    y = buf[y0:y0 + rows * N * 2].view(torch.bfloat16).view(rows, N)
    s0 = y0 - size + 16 if at == "last" else rows * N * 2 - 16
    scales = buf[s0:s0 + size]
    if kind == "e4m3":
        w = torch.zeros(2, N, K, device=DEV).to(torch.float8_e4m3fn)
        call = lambda: plan.expert_matmul(plan.new_rows8(rows, K), w, sp, y, w_scale=scales.view(torch.float32).view(2, N))
    else:
        w = torch.zeros(2, N, K // 8, dtype=torch.int32, device=DEV)
        x = torch.zeros(rows, K, dtype=torch.bfloat16, device=DEV)
        call = lambda: plan.expert_matmul_w4(x, w, scales.view(torch.bfloat16).view(2, N, K // 32), sp, y)
    with pytest.raises(A.A2avError, match="overlaps"):
        call()
    assert plan.launches == 0
    plan.close()


# ---- waits that run out ----------------------------------------------------------------

def gives_up_in_order(r, polls, K, swiglu):
    """With few polls a call ends, right or with its status bit; the next one, with the default, is right."""
    plan = r["plan"]
    plan.set_wait_limit(polls)
    for _ in range(3):
        r["call"]()
        status = plan.read_status(clear=True)
        assert status == A.DEV_WAIT_TIMEOUT or (polls > 0 and status == 0)
    plan.set_wait_limit(-1)
    r["y"].fill_(CANARY)
    r["call"]()
    assert plan.read_status() == 0
    for e, a, b in r["segs"]:
        within(r["y"][a:b], *product_ref(None, r["x64"][a:b], r["w64"][e], None, swiglu, K))
    plan.close()


@pytest.mark.parametrize("polls", [0, 1, 2, 3, 10, 100])
@pytest.mark.parametrize("counts", [[[0, 1030, 3, 2305]], [[1, 32, 0, 17]]], ids=["six stages", "ten stages"])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_pairs_give_up_in_order(kind, counts, polls):
    """Rings that go round, blocks of a pair that stop at different fills."""
    gives_up_in_order(run_product(kind, counts, 2576, 264, True, seed=polls), polls, 2576, True)


@pytest.mark.parametrize("polls", [0, 1, 2, 3, 10])
@pytest.mark.parametrize("K,swiglu", [(18432, False), (1024, True)])
def test_the_4bit_split_form_gives_up_in_order(K, swiglu, polls):
    gives_up_in_order(run_product("int4", [[1, 5, 0, 40]], K, 72, swiglu, group=64, seed=polls), polls, K, swiglu)


# ---- the norm's smallest and largest rows ------------------------------------------------

def both_norms(x, w, eps):
    """(y, rows8) of rows x [n][H]."""
    n, H = x.shape
    plan = A.Plan(1, 1, n, H, 1, device=DEV)
    y, rows8 = torch.full((1, n, H), CANARY, device=DEV, dtype=torch.bfloat16), plan.new_rows8((1, n), H).fill_(0xA5)
    plan.rms_norm(x.unsqueeze(0), w, y=y, rows8=rows8, eps=eps)
    torch.cuda.synchronize()
    plan.close()
    return y[0], rows8[0]


@pytest.mark.parametrize("H", [256, 512, 7168])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_norm_of_rows_with_subnormal_squares(H, eps):
    """Rows of 1e-20: a square is 71,000 steps of fp32's smallest, so it and the mean are half a step off each, 2^-16 of
    the value together, half of that in the root; the rest is 2^-18."""
    x = torch.full((3, H), 1e-20, device=DEV)
    x[1, ::2] *= -1
    x[2] = 1.0
    x, w = x.bfloat16(), (normal(gen(H), H) * 0.1 + 1).bfloat16()
    y, rows8 = both_norms(x, w, eps)
    _, v = norm_ref(x, None, w, eps)
    within(y, v, v.abs() * (BF + 2.0 ** -17 + 2.0 ** -18) + 1e-38)
    check_rows8(rows8, v, 2.0 ** -17 + 2.0 ** -18)


@pytest.mark.parametrize("H", [256, 512, 7168])
def test_norm_of_rows_at_the_end_of_the_range(H):
    """Squares up to 2^128 are right; past it the row is zeros, in y and in 8 bits, as the header says; with eps = 0 rows
    without a square have no norm."""
    g = gen(H)
    x = normal(g, 4, H)
    x[0, 3] = 1.8e19   # its square is 3.2e38
    x[1, 3] = 1.9e19   # 3.6e38, past 2^128
    x[2] = 0.0
    x[3] *= 1e15
    x, w = x.bfloat16(), torch.ones(H, device=DEV, dtype=torch.bfloat16)
    y, rows8 = both_norms(x, w, 1e-6)
    _, v = norm_ref(x, None, w, 1e-6)
    for row in (0, 2, 3):
        within(y[row], v[row], v[row].abs() * (BF + 2.0 ** -18) + 1e-38)
        if row != 2:
            check_rows8(rows8[row:row + 1], v[row:row + 1], 2.0 ** -18)
    for row in (1, 2):
        q, s = A.rows8_parts(rows8[row:row + 1])
        assert (y[row] == 0).all() and (q.float() == 0).all() and s == 0
    y, rows8 = both_norms(x, w, 0.0)
    assert torch.isnan(y[2]).all() and torch.isnan(A.rows8_parts(rows8[2:3])[1]).all()
