"""The norm and the experts' products against plain forms in 64 bits.

Tolerances, derived from the arithmetic (half a step: bf16 2^-8 of the value,
fp32 2^-24, e4m3 2^-4 of the value and 2^-10 of the scale below 2^-6 scales):

* norm: z is one fp32 sum (2^-24); v is z times two factors, each product
  rounded, the reciprocal root from a sum whose terms are all positive, in a
  tree of at most 4 + 5 + 5 sums after 16 fused ones: (16 + 14 + 8) * 2^-24 < 2^-18;
* a product's sum over K: each matrix instruction adds 16 terms (or 32 of 8
  bits), aligned to the largest and rounded, at most 2^-22 of the sum of
  magnitudes S each: (K/16 + 8) * 2^-22 * S, then half a bf16 step;
* SwiGLU: |d silu| <= 1.1 |dg|; exp and the division cost (8 + 2|g|) * 2^-23.
"""
import numpy as np
import pytest
import torch

import combine_device_resident_gb300 as A

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
BF = 2.0 ** -8
CANARY = 7.0


def gen(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def normal(g, *shape):
    return torch.randn(shape, generator=g, device=DEV)


def within(got, ref, tol):
    got, ref = got.double(), ref.double()
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float((got - ref).abs()[bad].max()), float(ref[bad].flatten()[0]),
                           float(got[bad].flatten()[0]))


# ---- the norm -------------------------------------------------------------------

def norm_ref(x, r, w, eps):
    z = x.double() + (r.double() if r is not None else 0.0)
    return z, z * torch.rsqrt(z.square().mean(-1, keepdim=True) + eps) * w.double()


def check_rows8(rows8, v, rel):
    """8-bit rows of v (fp64), v known to `rel`: the scale to that and a division, the values to half a
    step of e4m3, where a value near the middle of a step may fall to either side."""
    q, s = A.rows8_parts(rows8)
    a = v.abs().amax(-1)
    within(s, a / 448, a / 448 * (rel + 2.0 ** -22))
    unit = s.double().unsqueeze(-1)
    within(q.double() * unit, v, v.abs() * (2.0 ** -4 + 4 * rel) + unit * 2.0 ** -10)
    assert (rows8[..., -12:] == 0).all()


@pytest.mark.parametrize("R,T,H", [(1, 1, 8), (1, 1, 16), (2, 3, 256), (1, 5, 264), (4, 7, 5120), (2, 33, 7168),
                                   (1, 2, 8200), (1, 3, 16400), (1, 2, 32768), (32, 200, 48)])
@pytest.mark.parametrize("form", ["y", "rows8", "both", "alone"])
def test_norm(R, T, H, form):
    if form in ("rows8", "both") and H % 16:
        H += 8
    g = gen(R * 1000 + T * 10 + H)
    plan = A.Plan(R, R, T, H, 1, device=DEV)
    x = normal(g, R, T, H).bfloat16()
    r = None if form == "alone" else (normal(g, R, T, H) * 3).bfloat16()
    w = (normal(g, H) * 0.1 + 1).bfloat16()
    y = torch.full((R, T, H), CANARY, device=DEV, dtype=torch.bfloat16) if form != "rows8" else None
    rows8 = plan.new_rows8((R, T), H).fill_(0xA5) if form in ("rows8", "both") else None
    z = torch.empty_like(x) if r is not None else None
    plan.rms_norm(x, w, y=y, rows8=rows8, residual=r, residual_out=z, eps=1e-6)
    zr, v = norm_ref(x, r, w, 1e-6)
    if z is not None:
        within(z, zr, zr.abs() * (BF + 2.0 ** -23))
    if y is not None:
        within(y, v, v.abs() * (BF + 2.0 ** -18) + 1e-38)
    if rows8 is not None:
        check_rows8(rows8, v, 2.0 ** -18)
    assert plan.launches == 1
    plan.close()


@pytest.mark.parametrize("into", ["x", "residual"])
def test_norm_residual_in_place(into):
    g = gen(3)
    plan = A.Plan(2, 2, 70, 1040, 1, device=DEV)
    x, r = normal(g, 2, 70, 1040).bfloat16(), normal(g, 2, 70, 1040).bfloat16()
    w = normal(g, 1040).bfloat16()
    zr, v = norm_ref(x, r, w, 1e-5)
    y = torch.empty_like(x)
    out = x if into == "x" else r
    plan.rms_norm(x, w, y=y, residual=r, residual_out=out, eps=1e-5)
    within(out, zr, zr.abs() * (BF + 2.0 ** -23))
    within(y, v, v.abs() * (BF + 2.0 ** -18))
    plan.close()


def test_norm_special_rows():
    H = 512
    plan = A.Plan(1, 1, 8, H, 1, device=DEV)
    x = torch.ones(1, 8, H, device=DEV, dtype=torch.bfloat16)
    x[0, 0] = 0.0                      # a zero row
    x[0, 1, 3] = float("nan")          # NaN and infinities reach the scale
    x[0, 2, 5] = float("inf")
    x[0, 3] = 1e-20                    # tiny, lifted by eps = 0
    x[0, 4] = -2.0
    x[0, 5, 0] = 3e38                  # the squares overflow: v is 0, as in the plain form
    w = torch.ones(H, device=DEV, dtype=torch.bfloat16)
    y, rows8 = torch.empty_like(x), plan.new_rows8((1, 8), H)
    plan.rms_norm(x, w, y=y, rows8=rows8, eps=1e-6)
    q, s = A.rows8_parts(rows8)
    assert (y[0, 0] == 0).all() and s[0, 0] == 0 and (q[0, 0].float() == 0).all()
    assert torch.isnan(s[0, 1]) and torch.isnan(y[0, 1]).all() and torch.isnan(q[0, 1].float()).all()
    assert not torch.isfinite(s[0, 2])
    assert (y[0, 4] == -1).all()
    check_rows8(rows8[0, 4:5], norm_ref(x[0, 4:5], None, w, 1e-6)[1], 2.0 ** -18)
    assert (y[0, 5] == 0).all()
    assert (y[0, 6] == 1).all()        # neighbours are untouched by them
    plan.rms_norm(x, w, y=y, eps=0.0)
    zr, v = norm_ref(x[0, 3:5], None, w, 0.0)
    within(y[0, 4], v[1], v[1].abs() * (BF + 2.0 ** -18))
    plan.close()


def test_norm_active_tokens():
    R, T, H = 3, 5, 64
    g = gen(4)
    plan = A.Plan(R, R, T, H, 1, device=DEV)
    x, w = normal(g, R, T, H).bfloat16(), torch.ones(H, device=DEV, dtype=torch.bfloat16)
    y, rows8 = torch.full_like(x, CANARY), plan.new_rows8((R, T), H).fill_(0xA5)
    plan.set_active_tokens(torch.tensor([0, 2, 9], dtype=torch.int32, device=DEV))
    plan.rms_norm(x, w, y=y, rows8=rows8)
    _, v = norm_ref(x, None, w, 1e-6)
    for r, n in enumerate((0, 2, 5)):
        within(y[r, :n], v[r, :n], v[r, :n].abs() * (BF + 2.0 ** -18))
        assert (y[r, n:] == CANARY).all() and (rows8[r, n:] == 0xA5).all()
    plan.close()


# ---- layouts of dispatched rows ----------------------------------------------------

def layout(plan, counts):
    """Splits of rows grouped by expert, counts [R sources][E], and (expert, first row, end) of each."""
    R, E = counts.shape
    epr = E // R
    per = counts.reshape(R, R, epr).transpose(1, 2, 0)  # [d][le][source]
    first = np.cumsum(per.reshape(R, -1), 1).reshape(R, -1) - per.reshape(R, -1)
    total = per.reshape(R, -1).sum(1)
    fixed = plan.window_mode == "fixed"
    base = np.arange(R) * plan.window_rows if fixed else np.cumsum(total) - total
    sp = plan.new_splits()
    arrays = {"recv_total": total, "window_base": base, "recv_expert_counts": per.transpose(0, 2, 1)}
    if "recv_expert_offsets" in sp.names:
        arrays["recv_expert_offsets"] = first.reshape(R, epr, R).transpose(0, 2, 1)
    for n, v in arrays.items():
        getattr(sp, n).copy_(torch.from_numpy(np.ascontiguousarray(v, np.int32)))
    cap = plan.window_rows if fixed else 1 << 30
    segs = []
    for d in range(R):
        ends = np.cumsum(per[d].sum(1))
        for le in range(epr):
            lo, hi = min(ends[le] - per[d][le].sum(), cap), min(ends[le], cap)
            if hi > lo:
                segs.append((d * epr + le, int(base[d] + lo), int(base[d] + hi)))
    return sp, segs


def plan_for(counts, order="expert", window_rows=None):
    """A plan whose arena holds the rows of `counts` [R][E] (k = 1)."""
    R, E = counts.shape
    T = max(1, -(-int(counts.sum()) // R))
    kw = dict(window_mode="fixed", window_rows=window_rows) if window_rows else {}
    return A.Plan(R, E, T, 64, 1, device=DEV, recv_order=order, **kw)


def product_ref(kind, x, w, scale, swiglu, K):
    """fp64 (result, tolerance) of x [n][K] and w [Nw][K] as fp64 values."""
    p, S = x @ w.T, x.abs() @ w.abs().T
    e = (K / 16 + 8) * 2.0 ** -22 * S
    if not swiglu:
        return p, p.abs() * BF + e + 1e-38
    g, u = p.chunk(2, -1)
    eg, eu = e.chunk(2, -1)
    y = g * torch.sigmoid(g) * u
    return y, y.abs() * (BF + (8 + 2 * g.abs()) * 2.0 ** -23) + 1.1 * eg * u.abs() + g.abs() * eu + 1.1 * eg * eu + 1e-38


def run_product(kind, counts, K, N, swiglu, seed=0, order="expert", window_rows=None, group=32, poison=True, stream=None):
    g = gen(seed)
    counts = np.asarray(counts)
    plan = plan_for(counts, order, window_rows)
    sp, segs = layout(plan, counts)
    rows, E, Nw = plan.arena_rows, counts.shape[1], N * (2 if swiglu else 1)
    live = torch.zeros(rows, dtype=torch.bool, device=DEV)
    for _, a, b in segs:
        live[a:b] = True
    v = normal(g, rows, K)
    if poison:  # rows that are not live hold anything
        v[~live] = float("nan")
    w = normal(g, E, Nw, K) * K ** -0.5
    y = torch.full((rows, N), CANARY, device=DEV, dtype=torch.bfloat16)
    act = "swiglu" if swiglu else None
    if kind == "bf16":
        x, w = v.bfloat16(), w.bfloat16()
        x64, w64, ws = x.double(), w.double(), None
        call = lambda: plan.expert_matmul(x, w, sp, y, activation=act, stream=stream)
    elif kind == "e4m3":
        q, s = A.quantize_weights(v)
        x = plan.new_rows8(rows, K)
        xq, xs = A.rows8_parts(x)
        xq.copy_(q), xs.copy_(s)
        w8, ws = A.quantize_weights(w)
        x64, w64 = xq.double() * xs.double()[:, None], w8.double() * ws.double()[..., None]
        call = lambda: plan.expert_matmul(x, w8, sp, y, w_scale=ws, activation=act, stream=stream)
    else:
        x = v.bfloat16()
        w4, ws = A.pack_weights_w4(w, group)
        x64, w64 = x.double(), A.unpack_weights_w4(w4, ws).double()
        call = lambda: plan.expert_matmul_w4(x, w4, ws, sp, y, activation=act, stream=stream)
    torch.cuda.synchronize()
    call()
    torch.cuda.synchronize()
    assert plan.read_status() == 0
    for e, a, b in segs:
        ref, tol = product_ref(kind, x64[a:b], w64[e], ws, swiglu, K)
        within(y[a:b], ref, tol)
    assert (y[~live] == CANARY).all(), "a row that is not live was written"
    out = dict(plan=plan, sp=sp, segs=segs, x=x, y=y, call=call, x64=x64, w64=w64)
    return out


# one row; ragged ends around the 16- and 256-row tiles; experts without rows
COUNTS = {
    "one": [[0, 1]],
    "ragged": [[0, 1, 15, 16, 17, 0, 63, 65]],
    "tiles": [[255, 256, 257, 0]],
    "long": [[0, 1030, 3, 2305]],
    "ranks": [[1, 0, 2, 0, 5, 0, 0, 7], [3, 0, 0, 0, 1, 30, 0, 0], [0, 0, 9, 0, 0, 1, 0, 0], [0, 0, 4, 0, 2, 0, 0, 64]],
}


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("K,N", [(32, 8), (64, 64), (96, 136), (200, 72), (1040, 200), (2048, 256)])
@pytest.mark.parametrize("shape", list(COUNTS))
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int4"])
def test_products(kind, shape, K, N, swiglu):
    if kind == "e4m3":
        K = -(-K // 16) * 16
    if kind == "int4":
        K = -(-K // 32) * 32
    run_product(kind, COUNTS[shape], K, N, swiglu, seed=K + N)["plan"].close()


@pytest.mark.parametrize("most", [32, 33])
@pytest.mark.parametrize("kind", ["bf16", "e4m3"])
def test_either_ring(kind, most):
    """Up to 32 rows an expert the stages are smaller and more; enough of K to go round both rings."""
    run_product(kind, [[1, most, 0, 17, 5]], 2576, 264, True, seed=most)["plan"].close()


@pytest.mark.parametrize("kind,K", [("bf16", 8), ("e4m3", 16), ("int4", 32)])
def test_smallest_k(kind, K):
    run_product(kind, COUNTS["ragged"], K, 8, False)["plan"].close()


@pytest.mark.parametrize("group,K", [(64, 64), (64, 192), (128, 128), (128, 384), (128, 1920), (64, 2112)])
@pytest.mark.parametrize("swiglu", [False, True])
def test_w4_groups(group, K, swiglu):
    run_product("int4", COUNTS["ranks"], K, 104, swiglu, group=group, seed=group + K)["plan"].close()


def test_w4_many_items():
    counts = np.random.default_rng(5).integers(0, 5, (8, 64))
    run_product("int4", counts, 512, 1600, True, group=128)["plan"].close()  # items enough for the wide form
    run_product("int4", counts, 512, 2056, False, group=32)["plan"].close()


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("group,K,N", [(32, 32, 2568), (32, 160, 2568), (64, 64, 2560), (64, 832, 2600), (128, 128, 2560),
                                       (128, 1152, 2568)])
def test_w4_many_items_of_every_group(group, K, N, swiglu):
    counts = np.random.default_rng(group + K).integers(0, 4, (2, 64))
    counts[0, 3], counts[1, 5], counts[0, 6] = 45, 17, 16  # more rows than a work item, one more, as many
    run_product("int4", counts, K, N, swiglu, group=group, seed=K)["plan"].close()


def test_w4_many_items_in_fixed_windows():
    counts = np.random.default_rng(8).integers(0, 4, (4, 64))
    run_product("int4", counts, 256, 2568, True, group=64, window_rows=70)["plan"].close()


@pytest.mark.parametrize("swiglu", [False, True])
@pytest.mark.parametrize("group,K", [(32, 8224), (64, 10304), (128, 18432)])
def test_w4_few_items_of_long_rows(group, K, swiglu):
    """K past what a warp's boxes in flight hold (four of 256, eight warps), so that every ring goes round."""
    run_product("int4", [[1, 5, 0, 40]], K, 72, swiglu, group=group, seed=K)["plan"].close()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int4"])
@pytest.mark.parametrize("N", [72, 5128])
def test_more_live_rows_than_the_plan_has_tokens(kind, N, monkeypatch):
    """Splits of another plan's dispatch: every live row is computed, whatever the launch was sized for."""
    counts = np.array([[70, 0, 21, 1]])
    monkeypatch.setitem(globals(), "plan_for", lambda c, order, rows: A.Plan(
        1, 4, 1, 64, 1, device=DEV, window_mode="fixed", window_rows=rows, recv_order=order))
    run_product(kind, counts, 544, N, False, window_rows=96, seed=N)["plan"].close()


@pytest.mark.parametrize("items", [-1, 0, 1])
@pytest.mark.parametrize("swiglu", [False, True])
def test_w4_around_the_change_of_form(swiglu, items):
    """One expert whose items of 16 weight rows just fit on the SMs, two each, and one less and more."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    N = (2 * sms + items) * (8 if swiglu else 16)
    run_product("int4", [[3]], 288, N, swiglu, seed=N)["plan"].close()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int4"])
def test_all_experts_empty_and_most_experts(kind):
    r = run_product(kind, np.zeros((4, 16), int), 64, 64, False)
    assert (r["y"] == CANARY).all()
    r["plan"].close()
    counts = np.random.default_rng(1).integers(0, 3, (64, 2048)) * (np.random.default_rng(2).random((64, 2048)) < 0.02)
    run_product(kind, counts, 32, 16, True)["plan"].close()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int4"])
@pytest.mark.parametrize("window_rows", [40, 300])
def test_fixed_windows_and_overflow(kind, window_rows):
    counts = np.array([[3, 1, 0, 20, 0, 0, 9, 1], [0, 17, 5, 30, 1, 0, 0, 2]])
    run_product(kind, counts, 64, 72, False, window_rows=window_rows)["plan"].close()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int4"])
def test_one_expert_per_rank_in_source_order(kind):
    run_product(kind, np.array([[3, 40, 0], [1, 0, 0], [9, 2, 0]]), 64, 40, True, order="source")["plan"].close()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int4"])
def test_nan_stays_in_its_row_and_expert(kind):
    r = run_product(kind, [[5, 40, 0, 20]], 64, 64, False)
    clean = r["y"].clone()
    x = r["x"]
    if kind == "e4m3":
        x[7, 3] = 0x7F  # e4m3 NaN
    else:
        x[7, 3] = float("nan")
    r["call"]()
    torch.cuda.synchronize()
    assert torch.isnan(r["y"][7]).all()
    keep = [i for i in range(65) if i != 7]
    assert torch.equal(r["y"][keep], clean[keep])
    r["plan"].close()


@pytest.mark.parametrize("group", [32, 64, 128])
def test_nan_stays_in_its_row_with_many_items(group):
    r = run_product("int4", [[5, 40, 0, 20]], 256, 3600, False, group=group)
    clean = r["y"].clone()
    r["x"][7, 3] = float("nan")
    r["x"][9, 30] = float("inf")
    r["call"]()
    torch.cuda.synchronize()
    assert torch.isnan(r["y"][7]).all() and not torch.isfinite(r["y"][9]).any()
    keep = [i for i in range(65) if i not in (7, 9)]
    assert torch.equal(r["y"][keep], clean[keep])
    r["plan"].close()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int4"])
def test_infinite_sums_and_large_gates(kind):
    # gates far out on both sides: silu is 0 or the gate itself, never NaN
    plan = A.Plan(1, 1, 4, 64, 1, device=DEV, recv_order="expert")
    sp, _ = layout(plan, np.array([[4]]))
    K, N = 64, 8
    w = torch.zeros(1, 2 * N, K, device=DEV)
    w[0, :N, 0], w[0, N:, 1] = 7.0, 7.0
    v = torch.zeros(4, K, device=DEV)
    v[0, 0], v[1, 0], v[2, 0], v[3, 0] = 1000.0, -1000.0, 100.0, -100.0
    v[:, 1] = 1.0
    y = torch.zeros(4, N, device=DEV, dtype=torch.bfloat16)
    if kind == "bf16":
        plan.expert_matmul(v.bfloat16(), w.bfloat16(), sp, y, activation="swiglu")
    elif kind == "e4m3":
        x = plan.new_rows8(4, K)
        plan.quantize_rows(v.bfloat16(), sp, x)
        w8, ws = A.quantize_weights(w)
        plan.expert_matmul(x, w8, sp, y, w_scale=ws, activation="swiglu")
    else:
        w4, ws = A.pack_weights_w4(w, 32)
        plan.expert_matmul_w4(v.bfloat16(), w4, ws, sp, y, activation="swiglu")
    torch.cuda.synchronize()
    up = 7.0 if kind != "e4m3" else float((A.rows8_parts(x)[0].double() * A.rows8_parts(x)[1].double()[:, None])[0, 1] * 7)
    assert y[1].abs().max() < 1e-30 and y[3].abs().max() < 1e-30
    want = torch.tensor([7000.0 * up], device=DEV, dtype=torch.float64)
    within(y[0], want.expand(N), want.abs() * (BF + 2.0 ** -4 * (kind == "e4m3")))
    plan.close()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int4"])
def test_repeated_calls_give_the_same_bits(kind):
    r = run_product(kind, COUNTS["ranks"], 1024, 264, True, group=128)
    first = r["y"].clone()
    for _ in range(5):
        r["y"].fill_(CANARY)
        r["call"]()
        assert torch.equal(r["y"], first)
    r["plan"].close()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int4"])
def test_on_another_stream(kind):
    s = torch.cuda.Stream(DEV)
    s.wait_stream(torch.cuda.current_stream(DEV))
    run_product(kind, COUNTS["ragged"], 256, 64, True, stream=s)["plan"].close()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int4"])
def test_graph_follows_the_splits(kind):
    """A captured product reads the sizes that are in memory when it is replayed."""
    a, b = np.array([[3, 0, 30, 7]]), np.array([[0, 20, 1, 19]])
    r = run_product(kind, a, 64, 64, False, poison=False)
    s = torch.cuda.Stream(DEV)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=s):
        c = torch.cuda.current_stream(DEV)
        assert c == s
        r["call"]()
    sp2, segs = layout(r["plan"], b)
    for n in sp2.names:
        getattr(r["sp"], n).copy_(getattr(sp2, n))
    r["y"].fill_(CANARY)
    graph.replay()
    torch.cuda.synchronize()
    for e, lo, hi in segs:
        ref, tol = product_ref(kind, r["x64"][lo:hi], r["w64"][e], None, False, 64)
        within(r["y"][lo:hi], ref, tol)
    r["plan"].close()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int4"])
def test_rows_past_two_gibibytes(kind):
    """Row offsets past 2^31 bytes: the last rows of a long arena of wide rows."""
    K, N, n = 2048, 1032, 1 << 21
    plan = A.Plan(1, 2, n, 64, 1, device=DEV, recv_order="expert")
    sp, segs = layout(plan, np.array([[n - 37, 37]]))
    sp.recv_expert_offsets[0, 0, 0] = n - 37 - 5  # the first expert: only its last five rows
    sp.recv_expert_offsets[0, 0, 1] = n - 37
    g = gen(9)
    tail = normal(g, 42, K)
    w = normal(g, 2, N, K) * K ** -0.5
    y = torch.empty((n, N), device=DEV, dtype=torch.bfloat16)
    if kind == "e4m3":
        x = torch.empty((n, K + 16), device=DEV, dtype=torch.uint8)
        q, s = A.quantize_weights(tail)
        xq, xs = A.rows8_parts(x[-42:])
        xq.copy_(q), xs.copy_(s)
        w8, ws = A.quantize_weights(w)
        x64, w64 = xq.double() * xs.double()[:, None], w8.double() * ws.double()[..., None]
        plan.expert_matmul(x, w8, sp, y, w_scale=ws)
    else:
        x = torch.empty((n, K), device=DEV, dtype=torch.bfloat16)
        x[-42:] = tail.bfloat16()
        x64 = x[-42:].double()
        if kind == "bf16":
            plan.expert_matmul(x, w.bfloat16(), sp, y)
            w64 = w.bfloat16().double()
        else:
            w4, ws = A.pack_weights_w4(w, 128)
            w64 = A.unpack_weights_w4(w4, ws).double()
            plan.expert_matmul_w4(x, w4, ws, sp, y)
    for e, lo, hi in ((0, 0, 5), (1, 5, 42)):
        ref, tol = product_ref(kind, x64[lo:hi], w64[e], None, False, K)
        within(y[n - 42 + lo:n - 42 + hi], ref, tol)
    assert plan.read_status() == 0
    plan.close()


# ---- rows to 8 bits ------------------------------------------------------------------

@pytest.mark.parametrize("K", [16, 48, 1024, 2064, 16400])
@pytest.mark.parametrize("window_rows", [None, 12, 100])
def test_quantize_rows(K, window_rows):
    g = gen(K)
    counts = np.array([[3, 1, 0, 20], [0, 17, 5, 0]])
    plan = plan_for(counts, window_rows=window_rows)
    sp, segs = layout(plan, counts)
    x = normal(g, plan.arena_rows, K).bfloat16()
    rows8 = plan.new_rows8(plan.arena_rows, K).fill_(0xA5)
    plan.quantize_rows(x, sp, rows8)
    live = torch.zeros(plan.arena_rows, dtype=torch.bool, device=DEV)
    for _, a, b in segs:
        live[a:b] = True
    check_rows8(rows8[live], x[live].double(), 2.0 ** -22)
    assert (rows8[~live] == 0xA5).all()
    plan.close()


# ---- refusals on a real plan ------------------------------------------------------------

def test_refusals():
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device=DEV)
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8, device=DEV)
    plan = A.Plan(2, 4, 8, 64, 1, device=DEV, recv_order="expert")
    src = A.Plan(2, 4, 8, 64, 1, device=DEV)
    pad = A.Plan(2, 4, 8, 64, 1, window_mode="padded", device=DEV)
    odd = A.Plan(2, 4, 8, 72, 1, device=DEV)
    big = A.Plan(1, 1, 1, 32776, 1, device=DEV)
    sp, x, w, y = plan.new_splits(), bf(16, 64), bf(4, 16, 64), bf(16, 16)
    t, wt = bf(2, 8, 64), bf(64)
    f8 = torch.zeros(4, 16, 24, device=DEV).to(torch.float8_e4m3fn)
    i4 = lambda k: torch.zeros(4, 16, k // 8, dtype=torch.int32, device=DEV)
    cases = [
        (lambda: plan.rms_norm(t, wt), "neither"),
        (lambda: plan.rms_norm(t, wt, y=bf(2, 8, 64), residual_out=bf(2, 8, 64)), "without residual"),
        (lambda: plan.rms_norm(t, wt, y=bf(2, 8, 64), eps=-1.0), "eps"),
        (lambda: plan.rms_norm(t, wt, y=bf(2, 8, 64), eps=float("nan")), "eps"),
        (lambda: plan.rms_norm(t, wt, y=t), "overlaps an input"),
        (lambda: odd.rms_norm(bf(2, 8, 72), bf(72), rows8=u8(2, 8, 88)), "H % 16"),
        (lambda: big.rms_norm(bf(1, 1, 32776), bf(32776), y=bf(1, 1, 32776)), "32768"),
        (lambda: src.expert_matmul(x, w, src.new_splits(), y), "grouped by expert"),
        (lambda: pad.expert_matmul(bf(pad.arena_rows, 64), w, pad.new_splits(), bf(pad.arena_rows, 16)), "padded"),
        (lambda: pad.quantize_rows(bf(pad.arena_rows, 64), pad.new_splits(), u8(pad.arena_rows, 80)), "padded"),
        (lambda: plan.expert_matmul(x, bf(4, 12, 64), sp, bf(16, 12)), "N must"),
        (lambda: plan.expert_matmul(bf(16, 60), bf(4, 16, 60), sp, y), "K must"),
        (lambda: plan.expert_matmul(u8(16, 40), f8, sp, y, w_scale=torch.zeros(4, 16, device=DEV)), "K must"),
        (lambda: plan.expert_matmul(u8(16, 40), f8, sp, y), "pointer"),
        (lambda: plan.expert_matmul(x, w, sp, y, w_scale=torch.zeros(4, 16, device=DEV)), "no scales"),
        (lambda: plan.expert_matmul(x, bf(4, 64, 64), sp, x), "overlaps"),
        (lambda: plan.expert_matmul_w4(x, i4(64), bf(4, 16, 4), sp, y), "group"),
        (lambda: plan.quantize_rows(bf(16, 24), sp, u8(16, 40)), "multiple of 16"),
        (lambda: plan.expert_matmul(x.cpu(), w, sp, y), "is on"),
    ]
    for i, (call, message) in enumerate(cases):
        with pytest.raises(A.A2avError, match=message):
            call()
    buf = bf(16 * 64 + 8)
    with pytest.raises(A.A2avError, match="misaligned"):
        plan.expert_matmul(buf[4:4 + 16 * 64].view(16, 64), w, sp, y)
    for p in (plan, src, pad, odd, big):
        assert p.launches == 0
        p.close()


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int4"])
def test_waits_that_run_out_set_the_status(kind):
    r = run_product(kind, COUNTS["long"], 1024, 264, True)
    plan = r["plan"]
    plan.set_wait_limit(0)
    r["call"]()
    assert plan.read_status(clear=True) == A.DEV_WAIT_TIMEOUT
    plan.set_wait_limit(-1)
    r["y"].fill_(CANARY)
    r["call"]()
    assert plan.read_status() == 0
    for e, a, b in r["segs"]:
        ref, tol = product_ref(kind, r["x64"][a:b], r["w64"][e], None, True, 1024)
        within(r["y"][a:b], ref, tol)
    plan.close()


@pytest.mark.parametrize("polls", [0, 1, 3])
def test_waits_that_run_out_with_many_items(polls):
    counts = np.random.default_rng(3).integers(0, 4, (2, 64))
    r = run_product("int4", counts, 512, 2568, True, group=128)
    plan = r["plan"]
    plan.set_wait_limit(polls)
    r["call"]()
    assert plan.read_status(clear=True) in ((A.DEV_WAIT_TIMEOUT,) if polls == 0 else (0, A.DEV_WAIT_TIMEOUT))
    plan.set_wait_limit(-1)
    r["y"].fill_(CANARY)
    r["call"]()
    assert plan.read_status() == 0
    for e, a, b in r["segs"]:
        ref, tol = product_ref("int4", r["x64"][a:b], r["w64"][e], None, True, 512)
        within(r["y"][a:b], ref, tol)
    plan.close()
