"""The norms around a block and their gradient against the definition in 64 bits.

Tolerances.  A root of a mean: squares in a thread's row of at most 32, a tree of 5 + 5, a
division and a root: below 2^-18 of it.  z has two terms, each off by their factors'
roundings: e_z = 2^-18 |b g u| + 2^-22 |a residual| + 2^-23 |z|.  The second root
sees that error through the mean of squares: relative 2 sqrt(sum e_z^2 / sum z^2) + 2^-18,
and v = z w r2 both.  Outputs in bf16 add 2^-8 of themselves.

Gradient: every formula is evaluated with its terms' magnitudes in place of the
terms ("size"); a term passes through at most three sums of 38 roundings and some 60 products, additions
and quotients: 200 * 2^-24 < 2^-16, twice that where the second root's error (e_z above) enters through
cancelling terms of z: the factor 1 + rho, rho = sqrt(sum (|a res| + |b g u|)^2 / sum z^2).
Sums over tokens add their number in turn.
"""
import pytest
import torch

import combine_device_resident_gb300 as A

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
BF = 2.0 ** -8
CANARY = 7.0


def within(got, ref, tol):
    got, ref = got.double(), ref.double()
    bad = ~((got - ref).abs() <= tol)
    assert not bad.any(), (int(bad.sum()), float((got - ref).abs()[bad].max()), float(ref[bad].flatten()[0]),
                           float(got[bad].flatten()[0]))


def inputs(R, T, H, post=True, gate="channel", seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + H)

    def half(*shape, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device=DEV) * std + mean).bfloat16()

    lead = {"none": None, "channel": (), "rank": (R,), "token": (R, T)}[gate]
    return dict(x=half(R, T, H, std=0.7), residual=half(R, T, H, std=3.0), weight=half(H, std=0.1, mean=1.0),
                post_weight=half(H, std=0.1, mean=1.0) if post else None,
                gate=None if lead is None else half(*lead, H, std=0.3, mean=0.4),
                d_y=half(R, T, H), d_residual_out=half(R, T, H))


def wide(gate):
    return 1.0 if gate is None else gate.double().unsqueeze(1) if gate.dim() == 2 else gate.double()


def reference(i, alpha, beta, eps=1e-6):
    x, res, g = i["x"].double(), i["residual"].double(), wide(i["gate"])
    r1 = torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) if i["post_weight"] is not None else torch.ones_like(x[..., :1])
    u = x * r1 * i["post_weight"].double() if i["post_weight"] is not None else x
    z = alpha * res + beta * g * u
    size_z = (alpha * res).abs() + (beta * g * u).abs()
    e_z = 2.0 ** -18 * (beta * g * u).abs() + 2.0 ** -22 * (alpha * res).abs() + 2.0 ** -23 * z.abs()
    r2 = torch.rsqrt(z.square().mean(-1, keepdim=True) + eps)
    sum_z = (z.square().sum(-1, keepdim=True) + eps * z.shape[-1]).clamp(min=1e-300)
    off2 = 2 * (e_z.square().sum(-1, keepdim=True) / sum_z).sqrt() + 2.0 ** -18
    rho = (size_z.square().sum(-1, keepdim=True) / sum_z).sqrt()
    return dict(x=x, r1=r1, u=u, z=z, e_z=e_z, r2=r2, off2=off2, rho=rho, g=g, size_z=size_z)


def check_rows8(rows8, v, e_v):
    """8-bit rows of v, known to e_v: the scale to that of the largest and a division, the values to half a step."""
    q, s = A.rows8_parts(rows8)
    a = v.abs().amax(-1)
    within(s, a / 448, (e_v.amax(-1) + a * 2.0 ** -22) / 448)
    unit = s.double().unsqueeze(-1)
    rel = (e_v.amax(-1) / a.clamp(min=1e-30)).unsqueeze(-1) + 2.0 ** -21
    within(q.double() * unit, v, v.abs() * (2.0 ** -4 + 2 * rel) + unit * 2.0 ** -10 + 2 * e_v)
    assert (rows8[..., -12:] == 0).all()


def check(i, alpha, beta, residual_out=None, y=None, rows8=None, eps=1e-6, live=None):
    f = reference(i, alpha, beta, eps)
    part = torch.ones(f["z"].shape[:2], dtype=torch.bool, device=DEV) if live is None else live
    if residual_out is not None:
        within(residual_out[part], f["z"][part], (f["z"].abs() * BF + f["e_z"] * 1.01)[part])
    if y is None and rows8 is None:
        return
    w = i["weight"].double()
    v = f["z"] * f["r2"] * w
    e_v = v.abs() * (f["off2"] + 2.0 ** -22) + f["e_z"] * (f["r2"] * w).abs()
    if y is not None:
        within(y[part], v[part], (v.abs() * BF + e_v * 1.01 + 1e-38)[part])
    if rows8 is not None:
        check_rows8(rows8[part], v[part], e_v[part])


SHAPES = [(1, 1, 8), (1, 1, 16), (2, 3, 256), (1, 5, 264), (4, 7, 5120), (2, 33, 7168), (1, 2, 8200), (1, 3, 16400),
          (1, 2, 32768), (32, 200, 48), (8, 1, 5120), (3, 130, 1040), (64, 3, 512)]


@pytest.mark.parametrize("R,T,H", SHAPES)
@pytest.mark.parametrize("form", ["y", "rows8", "both", "residual"])
@pytest.mark.parametrize("post,gate", [(True, "channel"), (False, "none"), (True, "rank"), (False, "token"), (True, "none"),
                                       (False, "channel")])
def test_block_norm(R, T, H, form, post, gate):
    if form in ("rows8", "both") and H % 16:
        H += 8
    plan = A.Plan(R, R, T, H, 1, device=DEV)
    i = inputs(R, T, H, post, gate)
    z = torch.full_like(i["x"], CANARY) if form != "rows8" else None
    y = torch.full_like(i["x"], CANARY) if form in ("y", "both") else None
    rows8 = plan.new_rows8((R, T), H).fill_(0xA5) if form in ("rows8", "both") else None
    plan.block_norm(i["x"], i["residual"], residual_out=z, weight=i["weight"] if form != "residual" else None, y=y,
                    rows8=rows8, post_weight=i["post_weight"], gate=i["gate"], residual_scale=0.75, branch_scale=-1.5)
    check(i, 0.75, -1.5, z, y, rows8)
    assert plan.launches == 1
    plan.close()


def test_as_the_plain_norm():
    """Without a post norm, gate and scales it is the norm with the residual's addition."""
    plan = A.Plan(4, 4, 33, 1040, 1, device=DEV)
    i = inputs(4, 33, 1040, False, "none")
    out = [[torch.empty_like(i["x"]), torch.empty_like(i["x"]), plan.new_rows8((4, 33), 1040)] for _ in range(2)]
    plan.block_norm(i["x"], i["residual"], residual_out=out[0][0], weight=i["weight"], y=out[0][1], rows8=out[0][2])
    plan.rms_norm(i["x"], i["weight"], residual=i["residual"], residual_out=out[1][0], y=out[1][1], rows8=out[1][2])
    assert torch.equal(out[0][0], out[1][0])
    within(out[0][1], out[1][1].double(), out[1][1].double().abs() * 2.0 ** -7)  # one step where the sums' orders differ
    plan.close()


@pytest.mark.parametrize("into", ["x", "residual"])
@pytest.mark.parametrize("H", [48, 1040, 7168])
def test_in_place(into, H):
    plan = A.Plan(2, 2, 170, H, 1, device=DEV)
    i = inputs(2, 170, H)
    was = dict(i, x=i["x"].clone(), residual=i["residual"].clone())
    y = torch.empty_like(i["x"])
    plan.block_norm(i["x"], i["residual"], residual_out=i[into], weight=i["weight"], y=y, post_weight=i["post_weight"],
                    gate=i["gate"], residual_scale=0.5)
    check(was, 0.5, 1.0, i[into], y)
    plan.close()


@pytest.mark.parametrize("H", [48, 512, 7168])
def test_special_rows(H):
    plan = A.Plan(1, 1, 9, H, 1, device=DEV)
    i = inputs(1, 9, H)
    i["x"][0, 0], i["residual"][0, 0] = 0.0, 0.0      # nothing at all
    i["x"][0, 1, 3] = float("nan")
    i["residual"][0, 2, 5] = float("inf")
    i["x"][0, 3], i["residual"][0, 3] = 1e-20, 1e-20
    i["x"][0, 4] = 0.0                                # a block that gave nothing
    i["residual"][0, 5] = 0.0
    y, z, rows8 = torch.empty_like(i["x"]), torch.empty_like(i["x"]), plan.new_rows8((1, 9), H)
    plan.block_norm(i["x"], i["residual"], residual_out=z, weight=i["weight"], y=y, rows8=rows8,
                    post_weight=i["post_weight"], gate=i["gate"])
    q, s = A.rows8_parts(rows8)
    assert (y[0, 0] == 0).all() and (z[0, 0] == 0).all() and s[0, 0] == 0 and (q[0, 0].float() == 0).all()
    assert torch.isnan(s[0, 1]) and torch.isnan(y[0, 1]).all()
    assert not torch.isfinite(s[0, 2])
    live = torch.ones(1, 9, dtype=torch.bool, device=DEV)
    live[0, 0:4] = False
    check(i, 1.0, 1.0, z, y, rows8, live=live)
    plan.close()


@pytest.mark.parametrize("H", [48, 1040])
def test_tokens_that_take_no_part_are_left(H):
    R, T = 4, 6
    plan = A.Plan(R, R, T, H, 1, device=DEV)
    n = torch.tensor([0, 4, 9, -1], dtype=torch.int32, device=DEV)
    plan.set_active_tokens(n)
    live = torch.arange(T, device=DEV).view(1, T) < n.view(R, 1)
    for gate in ("channel", "rank", "token"):
        i = inputs(R, T, H, gate=gate)
        y, z = torch.full_like(i["x"], CANARY), torch.full_like(i["x"], CANARY)
        rows8 = plan.new_rows8((R, T), H).fill_(0xA5)
        plan.block_norm(i["x"], i["residual"], residual_out=z, weight=i["weight"], y=y, rows8=rows8,
                        post_weight=i["post_weight"], gate=i["gate"])
        check(i, 1.0, 1.0, z, y, rows8, live=live)
        assert (y[~live] == CANARY).all() and (z[~live] == CANARY).all() and (rows8[~live] == 0xA5).all()
        # what is behind the batch may hold anything
        i["x"][~live], i["d_y"][~live] = float("nan"), float("nan")
        run_grad(plan, i, gate, live=live)
    plan.close()


# ---- the gradient -------------------------------------------------------------------

def run_grad(plan, i, gate, alpha=1.0, beta=1.0, use=("d_y", "d_residual_out"), params=True, live=None, in_place=False,
             scratch=None):
    R, T, H = plan.R, plan.T, plan.H
    d_y = i["d_y"].clone() if "d_y" in use else None
    dro = i["d_residual_out"].clone() if "d_residual_out" in use else None
    fill = dict(device=DEV, dtype=torch.float32)
    dw = torch.full((H,), CANARY, **fill) if params and d_y is not None else None
    dp = torch.full((H,), CANARY, **fill) if params and i["post_weight"] is not None else None
    dg = None
    if params and i["gate"] is not None:
        dg = torch.full(i["gate"].shape, CANARY, device=DEV, dtype=torch.bfloat16 if gate == "token" else torch.float32)
    d_x = d_y if in_place and d_y is not None else torch.full_like(i["x"], CANARY)
    d_res = dro if in_place and dro is not None else torch.full_like(i["x"], CANARY)
    given = dict(weight=i["weight"] if d_y is not None else None, post_weight=i["post_weight"], gate=i["gate"])
    plan.block_norm_grad(i["x"], i["residual"], d_x, d_res, d_y=d_y, d_residual_out=dro, d_weight=dw, d_post_weight=dp,
                         d_gate=dg, scratch=scratch if scratch is not None else plan.new_norm_scratch() if params else None,
                         residual_scale=alpha, branch_scale=beta, **given)
    got = dict(d_x=d_x, d_residual=d_res, d_weight=dw, d_post=dp, d_gate=dg)
    check_grad(i, got, alpha, beta, use, live)
    return got


def check_grad(i, got, alpha, beta, use, live=None):
    part = torch.ones(i["x"].shape[:2], dtype=torch.bool, device=DEV) if live is None else live
    clean = {n: torch.where(part.unsqueeze(-1), t, torch.zeros_like(t)) if t is not None and t.dim() == 3 and n != "gate" else t
             for n, t in i.items()}
    f = reference(clean, alpha, beta)
    m = part.unsqueeze(-1).double()
    zero = torch.zeros_like(f["z"])
    dy = clean["d_y"].double() * m if "d_y" in use else zero
    dr = clean["d_residual_out"].double() * m if "d_residual_out" in use else zero
    loose = 2.0 ** -15 * (1 + f["rho"])

    def both(fn):  # the value, and the same of magnitudes
        return fn(lambda t: t, -1.0), fn(torch.abs, 1.0)

    w, r1, r2, z, x, u = (clean["weight"].double(), f["r1"], f["r2"], f["z"], f["x"], f["u"])
    dz, dz_s = both(lambda a, s: a(dr) + r2 * a(dy * w) + s * a(z) * r2 ** 3 * (a(dy * w) * a(z)).mean(-1, keepdim=True))
    within(got["d_residual"][part], (alpha * dz)[part], ((alpha * dz).abs() * BF + loose * dz_s * abs(alpha) + 1e-37)[part])
    db, db_s = beta * dz, abs(beta) * dz_s
    g = f["g"]
    du, du_s = db * g, db_s * (g.abs() if torch.is_tensor(g) else g)
    if clean["post_weight"] is not None:
        p = clean["post_weight"].double()
        dx = r1 * du * p - x * r1 ** 3 * (du * p * x).mean(-1, keepdim=True)
        dx_s = r1 * du_s * p.abs() + x.abs() * r1 ** 3 * (du_s * p.abs() * x.abs()).mean(-1, keepdim=True)
    else:
        dx, dx_s = du, du_s
    within(got["d_x"][part], dx[part], (dx.abs() * BF + loose * dx_s + 1e-37)[part])
    turns = (part.numel() + 64) * 2.0 ** -24
    sums = {}
    if got["d_weight"] is not None:
        sums["d_weight"] = (dy * z * r2, (dy * r2).abs() * f["size_z"], (0, 1))
    if got["d_post"] is not None:
        sums["d_post"] = (du * x * r1, du_s * (x * r1).abs(), (0, 1))
    if got["d_gate"] is not None:
        dims = {1: (0, 1), 2: (1,), 3: ()}[got["d_gate"].dim()]
        sums["d_gate"] = (db * u, db_s * u.abs(), dims)
    for name, (value, size, dims) in sums.items():
        if dims:
            ref, tol = (value * m).sum(dims), (size * m * (loose + turns)).sum(dims)
            within(got[name], ref, tol + 1e-37)
        else:
            within(got[name][part], value[part], (value.abs() * BF + size * loose + 1e-37)[part])
    if live is not None:
        for name in ("d_x", "d_residual") + (("d_gate",) if got["d_gate"] is not None and got["d_gate"].dim() == 3 else ()):
            assert (got[name][~part] == CANARY).all()


GRAD_SHAPES = [(1, 1, 8), (1, 1, 16), (2, 3, 256), (1, 5, 264), (4, 7, 5120), (2, 200, 7168), (1, 2, 8200), (1, 3, 16384),
               (32, 200, 48), (8, 1, 5120), (3, 130, 1040), (64, 5, 512), (1, 700, 2048), (7, 61, 136)]


@pytest.mark.parametrize("R,T,H", GRAD_SHAPES)
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", ["none", "channel", "rank", "token"])
def test_gradient(R, T, H, post, gate):
    plan = A.Plan(R, R, T, H, 1, device=DEV)
    i = inputs(R, T, H, post, gate, 1)
    run_grad(plan, i, gate, 0.75, -1.5)
    assert plan.launches == 2
    plan.close()


@pytest.mark.parametrize("H", [48, 1040, 7168])
@pytest.mark.parametrize("use", [("d_y",), ("d_residual_out",), ("d_y", "d_residual_out")])
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("params", [True, False])
def test_gradient_of_one_output(H, use, post, params):
    plan = A.Plan(2, 2, 90, H, 1, device=DEV)
    run_grad(plan, inputs(2, 90, H, post, "rank", 2), "rank", 0.5, 1.25, use, params)
    plan.close()


@pytest.mark.parametrize("H", [48, 1040, 7168])
def test_gradient_in_place(H):
    plan = A.Plan(2, 2, 170, H, 1, device=DEV)
    run_grad(plan, inputs(2, 170, H, True, "token", 3), "token", in_place=True)
    plan.close()


def test_gradient_same_bits_every_time():
    plan = A.Plan(4, 4, 300, 1040, 1, device=DEV)
    i = inputs(4, 300, 1040, True, "rank")
    scratch = plan.new_norm_scratch()
    a, b = (run_grad(plan, i, "rank", scratch=scratch.fill_(fill)) for fill in (0, 255))
    assert all(torch.equal(a[n], b[n]) for n in a)
    plan.close()


def test_gradient_without_tokens_is_zero():
    plan = A.Plan(2, 2, 5, 264, 1, device=DEV)
    plan.set_active_tokens(torch.zeros(2, dtype=torch.int32, device=DEV))
    i = inputs(2, 5, 264, True, "rank")
    got = run_grad(plan, i, "rank", live=torch.zeros(2, 5, dtype=torch.bool, device=DEV))
    assert all((got[n] == 0).all() for n in ("d_weight", "d_post", "d_gate"))
    plan.close()


@pytest.mark.parametrize("post,gate", [(True, "channel"), (False, "rank"), (True, "token")])
def test_gradient_by_differences(post, gate):
    """Along random directions of x, residual and the weights: central differences in 64 bits of
    sum(d_y * y + d_residual_out * z), off by h^2 of the third derivative (below 1e-5 of the terms at h = 1e-4), against
    the kernel's gradients, off by their roundings to bf16."""
    R, T, H = 2, 6, 136
    plan = A.Plan(R, R, T, H, 1, device=DEV)
    i = inputs(R, T, H, post, gate, 4)
    got = run_grad(plan, i, gate)
    names = {"x": "d_x", "residual": "d_residual", "weight": "d_weight", "post_weight": "d_post", "gate": "d_gate"}

    def loss(j):
        f = reference(j, 1.0, 1.0)
        return (i["d_y"].double() * f["z"] * f["r2"] * j["weight"].double()).sum() + (i["d_residual_out"].double() * f["z"]).sum()

    for n, (name, d) in enumerate(names.items()):
        if i[name] is None:
            continue
        v = torch.randn(i[name].shape, generator=torch.Generator().manual_seed(n)).to(DEV).double()
        h = 1e-4
        up, down = (loss(dict(i, **{name: i[name].double() + s * h * v})) for s in (1, -1))
        mine = (got[d].double() * v).sum()
        size = (got[d].double().abs() * v.abs()).sum()
        assert abs(mine - (up - down) / (2 * h)) <= size * (2.0 ** -8 + 1e-5) + 1e-4
    plan.close()


def test_other_stream_and_graph():
    R, T, H = 4, 50, 1040
    plan = A.Plan(R, R, T, H, 1, device=DEV)
    i = inputs(R, T, H)
    y, z = torch.empty_like(i["x"]), torch.empty_like(i["x"])
    common = dict(weight=i["weight"], post_weight=i["post_weight"], gate=i["gate"])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    plan.block_norm(i["x"], i["residual"], residual_out=z, y=y, stream=s, **common)
    s.synchronize()
    check(i, 1.0, 1.0, z, y)
    got = dict(d_x=torch.empty_like(y), d_residual=torch.empty_like(y), d_weight=torch.empty(H, device=DEV),
               d_post=torch.empty(H, device=DEV), d_gate=torch.empty(H, device=DEV))
    scratch = plan.new_norm_scratch()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.block_norm(i["x"], i["residual"], residual_out=z, y=y, **common)
        plan.block_norm_grad(i["x"], i["residual"], got["d_x"], got["d_residual"], d_y=i["d_y"],
                             d_residual_out=i["d_residual_out"], d_weight=got["d_weight"], d_post_weight=got["d_post"],
                             d_gate=got["d_gate"], scratch=scratch, **common)
    i["x"].mul_(-0.5)
    for _ in range(3):
        graph.replay()
    check(i, 1.0, 1.0, z, y)
    check_grad(i, got, 1.0, 1.0, ("d_y", "d_residual_out"))
    plan.close()


@pytest.mark.parametrize("H", [48, 1040, 8200])
def test_gradient_of_tiny_rows(H):
    """Rows of some 1e-14 with eps = 0: the roots' cubes lie past fp32's range, the gradients do not."""
    plan = A.Plan(1, 1, 5, H, 1, device=DEV)
    i = inputs(1, 5, H, True, "channel", 6)
    i["x"], i["residual"] = i["x"] * 2.0 ** -46, i["residual"] * 2.0 ** -46
    d_x, d_res = torch.empty_like(i["x"]), torch.empty_like(i["x"])
    plan.block_norm_grad(i["x"], i["residual"], d_x, d_res, weight=i["weight"], d_y=i["d_y"], post_weight=i["post_weight"],
                         gate=i["gate"], residual_scale=2.0, branch_scale=2.0 ** -46, eps=0.0)
    x, res = i["x"].double().requires_grad_(), i["residual"].double().requires_grad_()
    f = reference(dict(i, x=x, residual=res), 2.0, 2.0 ** -46, eps=0.0)
    loss = (f["z"] * f["r2"] * i["weight"].double() * i["d_y"].double()).sum()
    for got, want in zip((d_x, d_res), torch.autograd.grad(loss, (x, res))):
        assert torch.isfinite(got).all()
        # each element within the roundings of its row's terms (header): 2^-15 and bf16's half step of the row's largest
        within(got, want, want.abs().amax(-1, keepdim=True) * (BF + 2.0 ** -13))
    plan.close()


def test_refusals():
    R, T, H = 1, 4, 64
    plan = A.Plan(R, R, T, H, 1, device=DEV)
    i = inputs(R, T, H)
    x, res, w = i["x"], i["residual"], i["weight"]
    out, d = torch.empty_like(x), torch.empty_like(x)
    f = torch.empty(H, device=DEV)
    room = torch.empty(T + 1, H, device=DEV, dtype=torch.bfloat16)
    shifted = room.flatten()[8:8 + x.numel()].view_as(x)
    odd = A.Plan(1, 1, 2, 24, 1, device=DEV)
    big = A.Plan(1, 1, 1, 16392, 1, device=DEV)
    bx = torch.zeros(1, 1, 16392, device=DEV, dtype=torch.bfloat16)
    huge = A.Plan(1, 1, 1, 32776, 1, device=DEV)
    hx = torch.zeros(1, 1, 32776, device=DEV, dtype=torch.bfloat16)
    ox, ow = torch.zeros(1, 2, 24, device=DEV, dtype=torch.bfloat16), torch.zeros(24, device=DEV, dtype=torch.bfloat16)
    for call, message in [
        (lambda: plan.block_norm(x, res), "no output"),
        (lambda: plan.block_norm(x, res, y=out), "weight goes with"),
        (lambda: plan.block_norm(x, res, residual_out=out, weight=w), "weight goes with"),
        (lambda: plan.block_norm(x, res, weight=w, y=x), "overlaps"),
        (lambda: plan.block_norm(x, res, weight=w, y=out, residual_out=out), "overlaps"),
        (lambda: plan.block_norm(room[:T].view_as(x), res, residual_out=shifted), "overlaps"),
        # a weight or a gate in the first row of what is written in place
        (lambda: plan.block_norm(x, res, residual_out=x, gate=x[0, 0]), "overlaps"),
        (lambda: plan.block_norm(x, res, residual_out=res, post_weight=res[0, 0]), "overlaps"),
        (lambda: plan.block_norm(x, res, residual_out=x, gate=x[0, :1].view(1, H)), "overlaps"),
        (lambda: plan.block_norm(x, res, residual_out=x, y=out, weight=x[0, 0]), "overlaps"),
        (lambda: plan.block_norm_grad(x, res, i["d_y"], d, d_y=i["d_y"], weight=i["d_y"][0, 0]), "overlaps"),
        (lambda: plan.block_norm(x, res, residual_out=room.flatten()[1:1 + x.numel()].view_as(x)), "misaligned"),
        (lambda: odd.block_norm(ox, ox, weight=ow, rows8=odd.new_rows8((1, 2), 24)), "H % 16"),
        (lambda: huge.block_norm(hx, hx, residual_out=torch.empty_like(hx)), "H <= 32768"),
        (lambda: big.block_norm_grad(bx, bx, torch.empty_like(bx), torch.empty_like(bx), d_residual_out=bx), "H <= 16384"),
        (lambda: plan.block_norm_grad(x, res, out, d), "neither"),
        (lambda: plan.block_norm_grad(x, res, out, d, d_y=i["d_y"]), "needs weight"),
        (lambda: plan.block_norm_grad(x, res, out, d, d_residual_out=i["d_y"], weight=w, d_weight=f,
                                      scratch=plan.new_norm_scratch()), "d_weight needs"),
        (lambda: plan.block_norm_grad(x, res, out, d, d_residual_out=i["d_y"], d_post_weight=f,
                                      scratch=plan.new_norm_scratch()), "d_post_weight needs"),
        (lambda: plan.block_norm_grad(x, res, out, d, d_y=i["d_y"], weight=w, d_weight=f), "scratch"),
        (lambda: plan.block_norm_grad(x, res, out, out, d_y=i["d_y"], weight=w), "overlaps"),
        (lambda: plan.block_norm_grad(x, res, x, d, d_y=i["d_y"], weight=w), "overlaps"),
        (lambda: plan.block_norm_grad(x, res, out, d, d_y=i["d_y"], weight=w, d_weight=f, d_post_weight=f,
                                      post_weight=w, scratch=plan.new_norm_scratch()), "overlaps"),
        (lambda: plan.block_norm_grad(x, res, out, d, d_y=i["d_y"], weight=w, d_weight=f,
                                      scratch=plan.new_norm_scratch()[:-16]), "scratch has shape"),
    ]:
        with pytest.raises(A.A2avError, match=message):
            call()
    assert plan.launches == 0
    for p in (plan, odd, big, huge):
        p.close()
