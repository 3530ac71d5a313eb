"""The router by scores and its gradient against the definition in 64 bits.

Ids are whole numbers: equal, also where choices are nearer than fp32 tells apart.

Tolerances of the gates, relative: an exponential of x costs 2 * 2^-23 and its
argument's rounding |x| * 2^-24 (the fast one, in the softmax's sum, 2^-22 and
1.5 |x| * 2^-24); sums are at most 32 terms in a row, then a tree of 5; two
quotients and a product.  With |x| at most S, the token's spread of logits where a
score counts: (3 S + 80) * 2^-24.

The gradient: val = scale * r * (d - sum d r) * (1 - s): every factor as above, the
difference bounded by its terms' magnitudes, and (softmax) one more sum of k.
"""
import numpy as np
import pytest
import torch

import combine_device_resident_gb300 as A

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
FMAX = torch.finfo(torch.float32).max
INF = float("inf")


def clean(l):
    l = l.double().cpu()
    return torch.where(torch.isnan(l), torch.tensor(-FMAX, dtype=torch.float64), l).clamp(-FMAX, FMAX) + 0.0


def scores(l, rule):
    return torch.sigmoid(l) if rule.score == 1 else torch.softmax(l, -1)


def choose(logits, bias, rule, k):
    """Ids by the rule, in 64 bits on the CPU."""
    l = clean(logits)
    E, G = l.shape[-1], rule.groups
    s = scores(l, rule)
    c = l if bias is None else s + bias.double().cpu()
    c = torch.where(torch.isnan(c), torch.tensor(-INF, dtype=torch.float64), c) + 0.0
    out = torch.full((*l.shape[:-1], k), -1, dtype=torch.int64)
    for at in np.ndindex(*l.shape[:-1]):
        keep = np.ones(G, bool)
        row = c[at].numpy()
        if rule.groups_kept < G:
            per = row.reshape(G, E // G)
            best = -np.sort(-per, axis=1, kind="stable")[:, :rule.group_best]
            if bias is None and rule.group_best == 2:
                order = np.argsort(-per, axis=1, kind="stable")[:, :2]
                best = np.take_along_axis(s[at].numpy().reshape(G, E // G), order, 1)
            with np.errstate(invalid="ignore"):
                value = best.sum(1)
            value = np.where(np.isnan(value), -INF, value)
            keep[:] = False
            keep[np.lexsort((np.arange(G), -value))[:rule.groups_kept]] = True
        ids = np.arange(E)[np.repeat(keep, E // G)]
        out[at] = torch.from_numpy(ids[np.lexsort((ids, -row[ids]))[:k]].copy())
    return out


def gates(logits, idx, rule):
    l = clean(logits)
    if rule.renormalize:  # from log scores, which do not vanish
        ls = -torch.log1p(torch.exp(-l.abs())) + l.clamp(max=0) if rule.score == 1 else l
        return torch.softmax(ls.gather(-1, idx), -1) * rule.scale
    return scores(l, rule).gather(-1, idx) * rule.scale


def spread(logits):
    """How far below its token's largest a logit counts, and how far from 0: past 104 an exponential is 0."""
    l = clean(logits)
    return (l.amax(-1, keepdim=True) - l).clamp(max=104).amax(-1, keepdim=True) + l.abs().clamp(max=104).amax(-1, keepdim=True)


def run(plan, logits, rule, bias=None):
    idx = torch.full((plan.R, plan.T, plan.k), -7, dtype=torch.int32, device=DEV)
    gate = torch.full((plan.R, plan.T, plan.k), -7.0, device=DEV)
    plan.route_scores(logits, idx, gate, rule, bias=bias)
    return idx, gate


def check(plan, logits, rule, bias=None):
    idx, gate = run(plan, logits, rule, bias)
    want = choose(logits, bias, rule, plan.k)
    assert torch.equal(idx.cpu().long(), want)
    g = gates(logits, want, rule)
    tol = g.abs() * (3 * spread(logits) + 80) * 2.0 ** -24 + 1e-37
    assert ((gate.cpu().double() - g).abs() <= tol).all()
    assert plan.read_status() == 0
    return idx, gate


def make(R, E, T, k, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    plan = A.Plan(R, E, T, 8, k, device=DEV)
    logits = torch.randn(R, T, E, generator=g, device=DEV) * 1.5
    bias = torch.round(torch.randn(E, generator=g, device=DEV) * 30) * 1e-3
    return plan, logits, bias


SHAPES = [(1, 1, 1, 1), (1, 2, 3, 2), (1, 6, 5, 3), (2, 10, 7, 10), (1, 100, 33, 7), (8, 128, 1, 1), (4, 256, 65, 8),
          (2, 2048, 3, 32), (32, 256, 5, 6), (1, 16, 40, 4), (4, 32, 9, 8), (1, 64, 130, 2), (16, 512, 4, 8),
          (1, 36, 11, 8), (2, 160, 21, 6)]


@pytest.mark.parametrize("R,E,T,k", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("renormalize", [False, True])
def test_choice_and_gates(R, E, T, k, score, biased, renormalize):
    plan, logits, bias = make(R, E, T, k, E + T)
    check(plan, logits, A.RouteRule(score=score, renormalize=renormalize, scale=2.5), bias if biased else None)
    plan.close()


@pytest.mark.parametrize("R,E,T,k,G,kept", [(4, 256, 65, 8, 8, 4), (1, 64, 33, 4, 4, 1), (2, 32, 17, 8, 8, 3),
                                            (1, 96, 20, 6, 6, 5), (1, 128, 9, 2, 64, 3), (1, 12, 30, 2, 6, 1),
                                            (2, 2048, 3, 32, 64, 2), (1, 128, 40, 8, 2, 1), (1, 16, 50, 1, 16, 4),
                                            (1, 160, 19, 8, 8, 3), (8, 256, 33, 6, 16, 2)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("best", [1, 2])
def test_groups(R, E, T, k, G, kept, score, biased, best):
    if E // G < best:
        pytest.skip("a group holds fewer")
    plan, logits, bias = make(R, E, T, k, E + G)
    check(plan, logits, A.RouteRule(score=score, groups=G, groups_kept=kept, group_best=best, renormalize=True),
          bias if biased else None)
    plan.close()


RULES = [A.RouteRule(score=s, groups=g, groups_kept=n, group_best=b, renormalize=r)
         for s in ("softmax", "sigmoid") for g, n, b in ((1, 1, 1), (4, 2, 1), (4, 2, 2)) for r in (False, True)]


@pytest.mark.parametrize("E,k", [(64, 6), (256, 8), (20, 3)])
@pytest.mark.parametrize("rule", RULES, ids=lambda r: f"{r.score}-{r.groups}-{r.group_best}-{r.renormalize}")
@pytest.mark.parametrize("biased", [False, True])
def test_ties_go_to_the_lower_id(E, k, rule, biased):
    plan, logits, bias = make(1, E, 9, k)
    logits[0, 0] = 0.0                                                   # a router before training
    logits[0, 1] = torch.arange(E, device=DEV) % 3 - 1.0
    logits[0, 2] = torch.where(torch.arange(E, device=DEV) % 2 == 0, 0.0, -0.0)
    logits[0, 3] = 60.0                                                  # saturated scores
    logits[0, 4] = torch.arange(E, device=DEV) % 2 * 2e-7 + 1.0          # neighbours in fp32
    logits[0, 5] = -100.0
    bias = torch.round(bias * 50) / 50                                   # equal biases, too
    check(plan, logits, rule, bias if biased else None)
    plan.close()


@pytest.mark.parametrize("E,k,groups,kept,best", [(64, 6, 1, 1, 1), (256, 8, 8, 4, 2), (256, 8, 4, 1, 1), (128, 2, 1, 1, 1),
                                                  (512, 8, 8, 4, 2), (30, 5, 1, 1, 1)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [None, "zero", "few"])
def test_logits_of_few_bits(E, k, groups, kept, best, score, bias):
    """Logits out of a product in bf16 meet ties in most tokens; a bias starts at zero, or holds a few values."""
    plan, logits, b = make(2, E, 37, k, 9)
    logits = logits.bfloat16().float()
    b = {None: None, "zero": torch.zeros_like(b), "few": torch.round(b * 20) / 20}[bias]
    check(plan, logits, A.RouteRule(score=score, groups=groups, groups_kept=kept, group_best=best), b)
    plan.close()


@pytest.mark.parametrize("seed", range(60))
def test_any_shape_and_rule(seed):
    """Seeded sizes, rules and inputs: widths around the kernels' limits, kept groups from one to all."""
    rng = np.random.default_rng(seed)
    E = int(rng.choice([4, 8, 12, 16, 20, 28, 32, 40, 44, 60, 64, 68, 100, 128, 132, 160, 192, 252, 256, 260, 320, 512]))
    R = int(rng.choice([r for r in (1, 2, 4) if E % r == 0]))
    groups = int(rng.choice([g for g in (1, 1, 2, 4, 8, 16) if E % g == 0]))
    kept = int(rng.integers(1, groups + 1))
    k = int(rng.integers(1, min(12, kept * E // groups) + 1))
    best = int(rng.integers(1, 3)) if E // groups > 1 else 1
    rule = A.RouteRule(score=str(rng.choice(["softmax", "sigmoid"])), groups=groups, groups_kept=kept, group_best=best,
                       renormalize=bool(rng.integers(2)), scale=float(rng.choice([1.0, 0.5, 2.5])))
    plan, logits, bias = make(R, E, int(rng.integers(1, 70)), k, seed)
    if rng.integers(3) == 0:
        logits = logits * 20
    idx, _ = check(plan, logits, rule, bias if rng.integers(2) else None)
    grad_check(plan, logits, idx, rule, seed)
    plan.close()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("groups,kept,best", [(1, 1, 1), (8, 3, 1), (8, 3, 2)])
def test_choices_nearer_than_fp32_tells_apart(score, groups, kept, best):
    """Choices that agree to some 1e-8, every token of them: the order is that of 64 bits."""
    E, k, T = 256, 8, 64
    g = torch.Generator().manual_seed(3)
    bias = torch.round(torch.randn(E, generator=g) * 30) * 1e-3
    if score == "sigmoid":
        c = 0.5 + torch.rand(T, 1, generator=g).double() * 0.2 + torch.zeros(T, E, dtype=torch.float64)
        logits = torch.logit(c - bias.double()).float()
    else:
        bias = bias * 0.03
        p = (1.0 / E + bias.double().mean() - bias.double()).clamp(min=1e-5)
        logits = (torch.log(p) + torch.randn(T, 1, generator=g).double()).float()
    plan = A.Plan(1, E, T, 8, k, device=DEV)
    check(plan, logits.view(1, T, E).to(DEV), A.RouteRule(score=score, groups=groups, groups_kept=kept, group_best=best),
          bias.to(DEV))
    plan.close()


@pytest.mark.parametrize("E,k", [(64, 6), (256, 8), (18, 3)])
@pytest.mark.parametrize("rule", RULES, ids=lambda r: f"{r.score}-{r.groups}-{r.group_best}-{r.renormalize}")
@pytest.mark.parametrize("mask", [None, "-inf", "lowest", "-1e9", "nan", "inf", "all"])
def test_masked_experts_and_special_logits(E, k, rule, mask):
    if E % rule.groups:
        rule = A.RouteRule(score=("softmax", "sigmoid")[rule.score], groups=2, groups_kept=1, renormalize=bool(rule.renormalize))
    plan, logits, bias = make(1, E, 10, k, 5)
    if mask:
        v = {"-inf": -INF, "lowest": -FMAX, "-1e9": -1e9, "nan": float("nan"), "inf": INF, "all": -INF}[mask]
        bias[torch.randperm(E, generator=torch.Generator().manual_seed(1))[:E if mask == "all" else E // 3].to(DEV)] = v
    l = logits[0]
    l[0, ::2] = -INF
    l[1, ::3] = float("nan")
    l[2] = -INF                       # a token whose mask leaves nothing
    l[3] = float("nan")
    l[4, 5] = INF
    l[5, [1, 7, 11]] = INF
    l[6, ::2] = -FMAX
    l[7] *= 1e30
    l[8, 3:] = -INF
    check(plan, logits, rule, bias if mask else None)
    plan.close()


def test_tokens_that_take_no_part_are_left():
    plan, logits, bias = make(4, 32, 6, 4)
    rule = A.RouteRule(score="sigmoid", groups=4, groups_kept=2, group_best=2)
    n = torch.tensor([0, 3, 9, -2], dtype=torch.int32, device=DEV)
    plan.set_active_tokens(n)
    idx, gate = run(plan, logits, rule, bias)
    want = choose(logits, bias, rule, 4)
    d_logits = torch.full_like(logits, 5.0)
    plan.route_scores_grad(logits, idx, gate, d_logits, rule)
    for r, m in enumerate((0, 3, 6, 0)):
        assert torch.equal(idx[r, :m].cpu().long(), want[r, :m])
        assert (idx[r, m:] == -7).all() and (gate[r, m:] == -7.0).all()
        assert (d_logits[r, m:] == 5.0).all() and (d_logits[r, :m] != 5.0).all()
    plan.close()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("offset", [1, 2, 4])
def test_logits_off_the_16_byte_lines(score, offset):
    plan, logits, bias = make(2, 64, 37, 6)
    room = torch.empty(logits.numel() + offset, device=DEV)
    off = room[offset:].view_as(logits).copy_(logits)
    rule = A.RouteRule(score=score, renormalize=True)
    a, b = check(plan, off, rule, bias), check(plan, logits, rule, bias)
    d1, d2 = torch.empty(logits.numel() + offset, device=DEV)[offset:].view_as(logits), torch.empty_like(logits)
    plan.route_scores_grad(off, a[0], b[1], d1, rule)
    plan.route_scores_grad(logits, a[0], b[1], d2, rule)
    assert torch.equal(d1, d2)
    plan.close()


def test_other_stream_and_graph():
    plan, logits, bias = make(8, 256, 40, 8)
    rule = A.RouteRule(score="sigmoid", groups=8, groups_kept=4, group_best=2, scale=2.5)
    want, wg = run(plan, logits, rule, bias)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    idx, gate = torch.zeros_like(want), torch.zeros_like(wg)
    s.wait_stream(torch.cuda.current_stream())
    plan.route_scores(logits, idx, gate, rule, bias=bias, stream=s)
    s.synchronize()
    assert torch.equal(idx, want) and torch.equal(gate, wg)
    d = torch.empty_like(logits)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.route_scores(logits, idx, gate, rule, bias=bias)
        plan.route_scores_grad(logits, idx, gate, d, rule)
    logits.mul_(-1.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(idx.cpu().long(), choose(logits, bias, rule, 8))
    d2 = torch.empty_like(logits)
    plan.route_scores_grad(logits, idx, gate, d2, rule)
    assert torch.equal(d, d2)
    plan.close()


def test_as_the_plain_router():
    """Softmax over all, renormalised over the chosen, is the softmax over the chosen."""
    plan, logits, _ = make(8, 128, 50, 4)
    idx, gate = run(plan, logits, A.RouteRule(score="softmax", renormalize=True))
    i2, g2 = torch.empty_like(idx), torch.empty_like(gate)
    plan.route(logits, i2, g2)
    assert torch.equal(idx, i2)
    assert ((gate - g2).abs() <= g2 * 2.0 ** -18).all()
    plan.close()


# ---- the gradient ------------------------------------------------------------------

def grad_check(plan, logits, idx, rule, seed=0):
    g = torch.Generator().manual_seed(seed)
    d = torch.randn(plan.R, plan.T, plan.k, generator=g)
    got = torch.full_like(logits, 9.0)
    plan.route_scores_grad(logits, idx, d.to(DEV), got, rule)
    l = clean(logits).requires_grad_()
    i = idx.cpu().long()
    if rule.renormalize:
        ls = torch.nn.functional.logsigmoid(l) if rule.score == 1 else l
        y = torch.softmax(ls.gather(-1, i), -1) * rule.scale
    else:
        y = scores(l, rule).gather(-1, i) * rule.scale
    (want,) = torch.autograd.grad((y * d.double()).sum(), l)
    # magnitudes of the terms: |scale| * r_j * (|d_j| + sum |d| r), the dense part p * sum p |d|
    with torch.no_grad():
        y = y.abs()
        part = y * d.double().abs() + (y / abs(rule.scale)) * (y * d.double().abs()).sum(-1, keepdim=True)
        size = torch.zeros_like(want).scatter_add_(-1, i, part)
        if rule.score == 0 and not rule.renormalize:
            size += scores(l, rule) * (y * d.double().abs()).sum(-1, keepdim=True)
        tol = size * (4 * spread(logits) + 160 + 2 * plan.k) * 2.0 ** -24 + 1e-37
        assert ((got.cpu().double() - want).abs() <= tol).all()
    return got, d


@pytest.mark.parametrize("R,E,T,k", SHAPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_gradient(R, E, T, k, score, renormalize):
    plan, logits, bias = make(R, E, T, k, 7)
    rule = A.RouteRule(score=score, renormalize=renormalize, scale=1.75)
    idx, _ = run(plan, logits, rule, bias)
    got, _ = grad_check(plan, logits, idx, rule)
    again = torch.empty_like(got)
    plan.route_scores_grad(logits, idx, grad_input(plan), again, rule)
    assert torch.equal(got, again)  # the same bits every time
    assert plan.read_status() == 0
    plan.close()


def grad_input(plan):
    return torch.randn(plan.R, plan.T, plan.k, generator=torch.Generator().manual_seed(0)).to(DEV)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_gradient_by_differences(score, renormalize):
    """Along a random direction v, <grad, v> is the slope of sum d * gates(l + t v): central differences in 64 bits,
    off by h^2/6 of the third derivative (at most 8 here per unit of scale, d and v^3) and 1e-15 / h."""
    plan, logits, _ = make(2, 32, 9, 4, 11)
    rule = A.RouteRule(score=score, renormalize=renormalize, scale=1.5)
    idx, _ = run(plan, logits, rule)
    got, d = grad_check(plan, logits, idx, rule)
    v = torch.randn(logits.shape, generator=torch.Generator().manual_seed(2)).double()
    h, l, i = 1e-4, logits.cpu().double(), idx.cpu().long()
    f = [(gates(l + s * h * v, i, rule) * d.double()).sum((-1)) for s in (1, -1)]
    slope = (f[0] - f[1]) / (2 * h)
    mine = (got.cpu().double() * v).sum(-1)
    bound = 1.5 * d.double().abs().sum(-1) * (8 * h * h * v.abs().amax(-1) ** 3 + 1e-10 + 40 * 2.0 ** -22 * v.abs().amax(-1))
    assert ((mine - slope).abs() <= bound).all()
    plan.close()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_gradient_of_repeated_and_bad_ids(score, renormalize):
    plan, logits, _ = make(1, 40, 6, 4, 2)
    rule = A.RouteRule(score=score, renormalize=renormalize)
    idx, _ = run(plan, logits, rule)
    idx[0, 1] = torch.tensor([3, 3, 7, 3], device=DEV)
    idx[0, 2] = 5
    grad_check(plan, logits, idx, rule)
    assert plan.read_status() == 0
    # a bad id contributes nothing: the others as if it were not there
    full = torch.empty_like(logits)
    bad = idx.clone()
    bad[0, 3, 1], bad[0, 3, 3] = -1, 40
    d = grad_input(plan)
    plan.route_scores_grad(logits, bad, d, full, rule)
    assert plan.read_status(clear=True) == A.DEV_BAD_EXPERT
    two = A.Plan(1, 40, 6, 8, 2, device=DEV)
    few, dd = torch.empty_like(logits), d[..., [0, 2]].contiguous()
    two.route_scores_grad(logits, idx[..., [0, 2]].contiguous(), dd, few, rule)
    assert torch.allclose(full[0, 3], few[0, 3], rtol=2.0 ** -16, atol=1e-9)
    bad[0, 4] = -1
    plan.route_scores_grad(logits, bad, d, full, rule)
    assert (full[0, 4] == 0).all()
    two.close()
    plan.close()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_gradient_of_special_logits(score, renormalize):
    plan, logits, _ = make(1, 32, 8, 4, 2)
    l = logits[0]
    l[0, ::2] = -INF
    l[1] = -INF
    l[2] = float("nan")
    l[3, 4] = INF
    l[4] = 200.0
    l[5] = -200.0
    rule = A.RouteRule(score=score, renormalize=renormalize)
    idx, _ = run(plan, logits, rule)
    got, _ = grad_check(plan, logits, idx, rule)
    assert torch.isfinite(got).all()
    plan.close()


@pytest.mark.parametrize("change,message", [
    (dict(groups=3), "groups"), (dict(groups=0), "groups"), (dict(groups=128), "groups"), (dict(groups=4, groups_kept=5), "kept"),
    (dict(groups=4, groups_kept=0), "kept"), (dict(group_best=3), "group_best"), (dict(groups=64, groups_kept=32, group_best=2), "group_best"),
    (dict(scale=INF), "scale"), (dict(scale=float("nan")), "scale"), (dict(groups=32, groups_kept=1), "distinct"),
])
def test_rules_that_cannot_be_followed_are_refused(change, message):
    plan, logits, _ = make(1, 64, 3, 4)
    idx, gate = torch.zeros(1, 3, 4, dtype=torch.int32, device=DEV), torch.zeros(1, 3, 4, device=DEV)
    for call in (lambda r: plan.route_scores(logits, idx, gate, r),
                 lambda r: plan.route_scores_grad(logits, idx, gate, torch.empty_like(logits), r)):
        with pytest.raises(A.A2avError, match=message):
            call(A.RouteRule(**change))
    bad = A.RouteRule()
    bad.score = 2
    with pytest.raises(A.A2avError, match="score"):
        plan.route_scores(logits, idx, gate, bad)
    assert plan.launches == 0
    plan.close()


def test_overlaps_are_refused():
    plan = A.Plan(1, 8, 4, 8, 8, device=DEV)
    logits = torch.randn(1, 4, 8, device=DEV)
    idx, gate = torch.zeros(1, 4, 8, dtype=torch.int32, device=DEV), torch.zeros(1, 4, 8, device=DEV)
    rule = A.RouteRule()
    with pytest.raises(A.A2avError, match="overlaps"):
        plan.route_scores(logits, idx, logits, rule)
    with pytest.raises(A.A2avError, match="overlaps"):
        plan.route_scores(logits, idx, idx.view(torch.float32), rule)
    with pytest.raises(A.A2avError, match="overlaps"):
        plan.route_scores_grad(logits, idx, gate, logits, rule)
    with pytest.raises(A.A2avError, match="overlaps"):
        plan.route_scores_grad(logits, idx, gate, gate, rule)
    plan.close()
