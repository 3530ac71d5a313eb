"""Cases of the router's scored choice with its gradient, of the combine's gradient, and of the
norms before and after a block with the gate and the residual's scale, forward and backward.

A case is one call on the shapes of an MoE block: R ranks of T tokens, E experts, top-k, hidden H.
"""
import functools
import math

import torch

own = False

EPS = 1e-6
LOW8 = 448.0  # largest finite e4m3 value
ROUTE, ROUTE_GRAD, COMBINE_GRAD, NORM, NORM_GRAD = "route", "route grad", "combine grad", "norm", "norm grad"
CHUNK = 4096  # tokens at a time where the plain forms would need too much memory


def listed():
    grouped = dict(E=256, k=8, score="sigmoid", bias=True, groups=8, kept=4, best=2, renorm=True, scale=2.5)
    wide = dict(E=128, k=2, score="softmax", bias=False, groups=1, kept=1, best=1, renorm=False, scale=1.0)
    return [
        # one decode step, a token per rank: latency counts
        dict(name="route 8x128 top-1", op=ROUTE, R=8, T=1, E=128, k=1, score="sigmoid", bias=True, groups=1, kept=1,
             best=1, renorm=False, scale=1.0),
        # a decode batch, an odd count per rank: 4 of 8 groups, top-8, renormalised and scaled
        dict(grouped, name="route 2040x256 groups", op=ROUTE, R=8, T=255),
        # the prefill batch of the largest workload
        dict(grouped, name="route 65536x256 groups", op=ROUTE, R=32, T=2048),
        # softmax over all experts, gates as they are, no groups: an odd prefill batch
        dict(wide, name="route 16336x128 softmax", op=ROUTE, R=16, T=1021),
        # training: the gates' gradient back to the logits
        dict(grouped, name="route grad 65536x256", op=ROUTE_GRAD, R=32, T=2048),
        # the same through the whole softmax: every logit of a token gets one
        dict(wide, name="route grad 16336x128 softmax", op=ROUTE_GRAD, R=16, T=1021),
        # a small top-1 batch, an odd count per rank
        dict(name="combine grad 2040x5120 top-1", op=COMBINE_GRAD, R=8, T=255, E=16, k=1, H=5120),
        # the largest workload's step
        dict(name="combine grad 65536x7168 top-8", op=COMBINE_GRAD, R=32, T=2048, E=256, k=8, H=7168),
        # one decode step between two blocks, the next one's rows in 8 bits: latency counts
        dict(name="norm 8x5120 to 8 bits", op=NORM, R=8, T=1, H=5120, post=True, gate="channel", bits=8, alpha=1.0,
             beta=0.5),
        # a prefill batch between two blocks
        dict(name="norm 65536x7168", op=NORM, R=32, T=2048, H=7168, post=True, gate="channel", bits=16, alpha=1.0,
             beta=0.5),
        # a small training batch, a gate for each rank's sequence
        dict(name="norm grad 2040x5120 rank gates", op=NORM_GRAD, R=8, T=255, H=5120, post=True, gate="rank",
             alpha=1.0, beta=1.0),
        # the largest training batch
        dict(name="norm grad 65536x7168", op=NORM_GRAD, R=32, T=2048, H=7168, post=True, gate="channel", alpha=1.0,
             beta=0.5),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _rule(rng, E, k):
    groups = rng.choice([g for g in (1, 1, 2, 4, 8) if E % g == 0])
    size = E // groups
    kept = rng.randint(-(-k // size), groups)
    return dict(score=rng.choice(["softmax", "sigmoid"]), bias=rng.random() < 0.5, groups=groups, kept=kept,
                best=rng.choice([1, 2]) if size > 1 else 1, renorm=k > 1 and rng.random() < 0.6,
                scale=rng.choice([1.0, 2.5]))


def draw(rng):
    op = rng.choice([ROUTE, ROUTE, ROUTE_GRAD, COMBINE_GRAD, NORM, NORM_GRAD])
    R = rng.choice([1, 2, 4, 8, 16, 32])
    if op in (NORM, NORM_GRAD):
        H = max(16, _log(rng, 256, 7168) // 16 * 16)
        c = dict(op=op, R=R, T=_log(rng, 1, max(1, 2 ** 29 // (H * R * 2))), H=H, post=rng.random() < 0.7,
                 gate=rng.choice(["none", "channel", "rank", "token"]), alpha=rng.choice([1.0, 0.7]),
                 beta=rng.choice([1.0, 0.5]))
        return dict(c, bits=rng.choice([8, 16])) if op == NORM else c
    E = R * rng.choice([1, 2, 4, 8])
    k = min(E, rng.choice([1, 2, 4, 6, 8]))
    c = dict(op=op, R=R, E=E, k=k)
    if op == COMBINE_GRAD:
        H = max(8, _log(rng, 256, 7168) // 8 * 8)
        return dict(c, T=_log(rng, 1, max(1, 2 ** 30 // (H * R * k))), H=H)
    return dict(c, T=_log(rng, 1, 65536 // R), **_rule(rng, E, k))


# ---- inputs -------------------------------------------------------------------

def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = (c["R"], c["T"])

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(std).add_(mean)

    def half(*shape, std=1.0, mean=0.0):
        return normal(*shape, std=std, mean=mean).to(torch.bfloat16)

    def zeros(*shape, dtype=torch.bfloat16):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    s = {"case": c}
    if c["op"] in (ROUTE, ROUTE_GRAD):
        # a router's logits, some experts liked more than others; its biases a few thousandths apart
        s["logits"] = normal(*n, c["E"], std=1.5).add_(normal(c["E"], std=0.5))
        s["bias"] = (normal(c["E"], std=30.0).round_() * 1e-3) if c["bias"] else None
        s["idx"] = zeros(*n, c["k"], dtype=torch.int32)
        s["gate"] = zeros(*n, c["k"], dtype=torch.float32)
        if c["op"] == ROUTE_GRAD:
            choice, _, _ = _choose(c, s["logits"], s["bias"])
            s["idx"].copy_(choice)
            s["d_gate"] = normal(*n, c["k"])
            s["d_logits"] = zeros(*n, c["E"], dtype=torch.float32)
        return s
    H = c["H"]
    if c["op"] == COMBINE_GRAD:
        R, T, E, k = c["R"], c["T"], c["E"], c["k"]
        # the rows as the dispatch lays them out: windows by destination, sources in order, sorted by expert
        idx = torch.rand(R, T, E, generator=g, device="cuda").argsort(-1)[..., :k]
        epr = E // R
        key = ((idx // epr) * R + torch.arange(R, device="cuda").view(R, 1, 1)) * epr + idx % epr
        order = key.flatten().argsort(stable=True)
        slot = torch.empty_like(order)
        slot[order] = torch.arange(order.numel(), device="cuda")
        s["slot_map"] = slot.view(R, T, k).to(torch.int32)
        s["gate"] = torch.softmax(normal(R, T, k), -1)
        s["d_out"] = half(*n, H, std=1e-2)
        s["y"] = torch.cat([half(min(1 << 16, R * T * k - a), H) for a in range(0, R * T * k, 1 << 16)])
        s["d_y"] = zeros(R * T * k, H)
        s["d_gate"] = zeros(R, T, k, dtype=torch.float32)
        return s
    # a block's output, the residual stream some layers deep; norms' weights lie near 1, gates start small
    s["x"], s["residual"] = half(*n, H, std=0.7), half(*n, H, std=3.0)
    s["weight"] = half(H, std=0.1, mean=1.0)
    s["post"] = half(H, std=0.1, mean=1.0) if c["post"] else None
    lead = {"none": None, "channel": (), "rank": n[:1], "token": n}[c["gate"]]
    s["g"] = None if lead is None else half(*lead, H, std=0.2, mean=0.4)
    if c["op"] == NORM:
        s["residual_out"] = zeros(*n, H)
        if c["bits"] == 8:  # K bytes of e4m3, the fp32 scale, padding to 16 bytes
            s["rows8"] = zeros(*n, H + 16, dtype=torch.uint8)
            s["q"] = s["rows8"][..., :H].view(torch.float8_e4m3fn)
            s["scale"] = s["rows8"][..., H:H + 4].view(torch.float32)[..., 0]
        else:
            s["y"] = zeros(*n, H)
        return s
    s["d_y"], s["d_residual_out"] = half(*n, H, std=1e-2), half(*n, H, std=1e-2)
    s["d_x"], s["d_residual"] = zeros(*n, H), zeros(*n, H)
    s["d_weight"] = zeros(H, dtype=torch.float32)
    s["d_post"] = zeros(H, dtype=torch.float32) if c["post"] else None
    kind = torch.bfloat16 if c["gate"] == "token" else torch.float32
    s["d_g"] = None if lead is None else zeros(*lead, H, dtype=kind)
    return s


# ---- the plain forms ----------------------------------------------------------

def _choose(c, logits, bias):
    """Ids in descending order of choice (ties to the lower id), in 64 bits: neighbours at the border
    are nearer to each other than 32 bits tell apart.  Also the scores in 32 and 64 bits."""
    l64 = logits.double()
    score64 = torch.sigmoid(l64) if c["score"] == "sigmoid" else torch.softmax(l64, -1)
    # without a bias the experts' order is the logits', which no score's rounding can tie
    choice = score64 + bias.double() if c["bias"] else l64
    G = c["groups"]
    if c["kept"] < G:
        shape = (*logits.shape[:-1], G, c["E"] // G)
        value = (choice if c["bias"] or c["best"] == 1 else score64).view(shape)
        value = value.sort(-1, descending=True).values[..., :c["best"]].sum(-1)
        kept = value.sort(dim=-1, descending=True, stable=True).indices[..., :c["kept"]]
        keep = torch.zeros(shape[:-1], dtype=torch.bool, device=logits.device).scatter_(-1, kept, True)
        choice = torch.where(keep.unsqueeze(-1), choice.view(shape), -math.inf).view(choice.shape)
    idx = choice.sort(dim=-1, descending=True, stable=True).indices[..., :c["k"]]
    l32 = logits.float()
    score = torch.sigmoid(l32) if c["score"] == "sigmoid" else torch.softmax(l32, -1)
    return idx, score, score64


def _gates(c, score, idx):
    g = score.gather(-1, idx.long())
    if c["renorm"]:
        g = g / g.sum(-1, keepdim=True)
    return g * c["scale"]


def _route_grad(c, logits, idx, d_gate):
    sigmoid = c["score"] == "sigmoid"
    score = torch.sigmoid(logits) if sigmoid else torch.softmax(logits, -1)
    idx, dg = idx.long(), d_gate * c["scale"]
    s = score.gather(-1, idx)
    if c["renorm"]:
        total = s.sum(-1, keepdim=True)
        dg = (dg - (dg * s).sum(-1, keepdim=True) / total) / total
    ds = torch.zeros_like(score).scatter_add_(-1, idx, dg)
    if sigmoid:
        return ds * score * (1.0 - score)
    return score * (ds - (ds * score).sum(-1, keepdim=True))


def _combine_grad(s):
    c = s["case"]
    H, k = c["H"], c["k"]
    slot, gate = s["slot_map"].view(-1, k).long(), s["gate"].view(-1, k)
    d_out = s["d_out"].view(-1, H)
    d_gate, d_y = torch.empty_like(gate), torch.empty_like(s["y"])
    for a in range(0, slot.shape[0], CHUNK):
        at, d = slot[a:a + CHUNK], d_out[a:a + CHUNK].float().unsqueeze(1)
        d_gate[a:a + CHUNK] = (s["y"][at].float() * d).sum(-1)
        d_y[at.flatten()] = (gate[a:a + CHUNK].unsqueeze(-1) * d).to(torch.bfloat16).view(-1, H)
    return {"d_y": d_y, "d_gate": d_gate.view(s["gate"].shape)}


def _gate_of(c, g):
    return 1.0 if g is None else g.float().unsqueeze(1) if c["gate"] == "rank" else g.float()


def _norm(c, x, residual, post, g):
    x = x.float()
    r1 = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) if c["post"] else 1.0
    n = x * r1
    u = n * post.float() if c["post"] else n
    z = c["alpha"] * residual.float() + c["beta"] * _gate_of(c, g) * u
    r2 = torch.rsqrt((z * z).mean(-1, keepdim=True) + EPS)
    return x, r1, n, u, z, r2


def _plain(s):
    c = s["case"]
    if c["op"] == ROUTE:
        idx, score, _ = _choose(c, s["logits"], s["bias"])
        return {"idx": idx.to(torch.int32), "gate": _gates(c, score, idx)}
    if c["op"] == ROUTE_GRAD:
        return _route_grad(c, s["logits"], s["idx"], s["d_gate"])
    if c["op"] == COMBINE_GRAD:
        return _combine_grad(s)
    x, r1, n, u, z, r2 = _norm(c, s["x"], s["residual"], s["post"], s["g"])
    if c["op"] == NORM:
        v = z * r2 * s["weight"].float()
        out = {"residual": z.to(torch.bfloat16)}
        if c["bits"] == 16:
            return dict(out, y=v.to(torch.bfloat16))
        peak = v.abs().amax(-1)
        q = (v * (LOW8 / peak).unsqueeze(-1)).clamp_(-LOW8, LOW8).to(torch.float8_e4m3fn)
        return dict(out, q=q, scale=peak / LOW8)
    dy = s["d_y"].float()
    dv = dy * s["weight"].float()
    dz = s["d_residual_out"].float() + r2 * dv - z * r2 ** 3 * (dv * z).mean(-1, keepdim=True)
    out = {"d_residual": (c["alpha"] * dz).to(torch.bfloat16), "d_weight": (dy * z * r2).sum((0, 1))}
    db = c["beta"] * dz
    if c["gate"] != "none":
        dg = db * u
        out["d_gate"] = {"channel": lambda: dg.sum((0, 1)), "rank": lambda: dg.sum(1),
                         "token": lambda: dg.to(torch.bfloat16)}[c["gate"]]()
    du = db * _gate_of(c, s["g"])
    if c["post"]:
        out["d_post"] = (du * n).sum((0, 1))
        dn = du * s["post"].float()
        du = r1 * dn - x * r1 ** 3 * (dn * x).mean(-1, keepdim=True)
    return dict(out, d_x=du.to(torch.bfloat16))


# ---- the framework's calls ----------------------------------------------------

@functools.lru_cache(maxsize=None)
def _plan(R, E, T, H, k):
    import combine_device_resident_gb300 as a2av

    return a2av.Plan(R, E, T, H, k, device="cuda:0")


def _own(s):
    import combine_device_resident_gb300 as a2av

    c = s["case"]
    if "plan" not in s:
        s["plan"] = _plan(c["R"], c.get("E", c["R"]), c["T"], c.get("H", 8), c.get("k", 1))
    plan = s["plan"]
    if c["op"] in (ROUTE, ROUTE_GRAD):
        if "rule" not in s:
            s["rule"] = a2av.RouteRule(score=c["score"], groups=c["groups"], groups_kept=c["kept"],
                                       group_best=c["best"], renormalize=c["renorm"], scale=c["scale"])
        if c["op"] == ROUTE:
            plan.route_scores(s["logits"], s["idx"], s["gate"], s["rule"], bias=s["bias"])
            return {"idx": s["idx"], "gate": s["gate"]}
        plan.route_scores_grad(s["logits"], s["idx"], s["d_gate"], s["d_logits"], s["rule"])
        return s["d_logits"]
    if c["op"] == COMBINE_GRAD:
        plan.combine_grad(s["d_out"], s["y"], s["gate"], s["slot_map"], d_y=s["d_y"], d_gate=s["d_gate"])
        return {"d_y": s["d_y"], "d_gate": s["d_gate"]}
    common = dict(weight=s["weight"], post_weight=s["post"], gate=s["g"], residual_scale=c["alpha"],
                  branch_scale=c["beta"], eps=EPS)
    if c["op"] == NORM:
        plan.block_norm(s["x"], s["residual"], residual_out=s["residual_out"], y=s.get("y"), rows8=s.get("rows8"),
                        **common)
        out = {"residual": s["residual_out"]}
        return dict(out, y=s["y"]) if c["bits"] == 16 else dict(out, q=s["q"], scale=s["scale"])
    if "scratch" not in s:
        s["scratch"] = plan.new_norm_scratch()
    plan.block_norm_grad(s["x"], s["residual"], s["d_x"], s["d_residual"], d_y=s["d_y"],
                         d_residual_out=s["d_residual_out"], d_weight=s["d_weight"], d_post_weight=s["d_post"],
                         d_gate=s["d_g"], scratch=s["scratch"], **common)
    out = {"d_residual": s["d_residual"], "d_weight": s["d_weight"]}
    if c["gate"] != "none":
        out["d_gate"] = s["d_g"]
    if c["post"]:
        out["d_post"] = s["d_post"]
    return dict(out, d_x=s["d_x"])


def run(s):
    return _own(s) if own else _plain(s)


# ---- what a pass cannot do without ---------------------------------------------

def work(c):
    n = c["R"] * c["T"]
    if c["op"] in (ROUTE, ROUTE_GRAD):
        E, k = c["E"], c["k"]
        if c["op"] == ROUTE:
            return {"bytes": n * (4 * E + 8 * k) + (4 * E if c["bias"] else 0), "flops": 4 * n * E}
        # without the whole softmax only the chosen logits matter
        dense = c["score"] == "softmax" and not c["renorm"]
        return {"bytes": n * (4 * E + 8 * k + (4 * E if dense else 4 * k)), "flops": n * (4 * E if dense else 8 * k)}
    H = c["H"]
    if c["op"] == COMBINE_GRAD:
        k = c["k"]
        return {"bytes": n * (2 * H + k * (4 * H + 12)), "flops": 3 * n * k * H}
    gates = {"none": 0, "channel": 1, "rank": c["R"], "token": n}[c["gate"]]
    weights = 2 if c["post"] else 1
    if c["op"] == NORM:
        row = 6 * H + (H + 4 if c["bits"] == 8 else 2 * H)
        return {"bytes": n * row + 2 * H * (gates + weights), "flops": 12 * n * H}
    return {"bytes": n * 12 * H + H * (6 * weights + (4 if c["gate"] == "token" else 6) * gates), "flops": 30 * n * H}


# ---- the definition in 64 bits --------------------------------------------------

def _exact_route(c, s):
    E, k, G = c["E"], c["k"], c["groups"]
    l = s["logits"].to(torch.float64).view(-1, E)
    if c["score"] == "sigmoid":
        score = 1.0 / (1.0 + torch.exp(-l))
    else:
        e = torch.exp(l - l.amax(-1, keepdim=True))
        score = e / e.sum(-1, keepdim=True)
    if c["op"] == ROUTE:
        left = score + s["bias"].to(torch.float64) if c["bias"] else l.clone()
        low = torch.tensor(-math.inf, dtype=torch.float64, device="cuda")
        if c["kept"] < G:
            per = (left if c["bias"] or c["best"] == 1 else score).view(-1, G, E // G)
            value = per.amax(-1)
            if c["best"] == 2:
                first = (per == value.unsqueeze(-1)).to(torch.int8).argmax(-1, keepdim=True)
                value = value + per.scatter(-1, first, -math.inf).amax(-1)
            ids = torch.arange(G, device="cuda")
            # a group stays if fewer than `kept` go before it
            before = (value.unsqueeze(-2) > value.unsqueeze(-1)) | (
                (value.unsqueeze(-2) == value.unsqueeze(-1)) & (ids.view(1, G) < ids.view(G, 1)))
            keep = before.sum(-1) < c["kept"]
            left = torch.where(keep.repeat_interleave(E // G, dim=-1), left, low)
        ids, picks = torch.arange(E, device="cuda"), []
        for _ in range(k):
            best = torch.where(left == left.amax(-1, keepdim=True), ids, E).amin(-1, keepdim=True)
            picks.append(best)
            left = left.scatter(-1, best, -math.inf)
        idx = torch.cat(picks, -1)
        chosen = torch.take_along_dim(score, idx, -1)
        if c["renorm"]:
            chosen = chosen / chosen.sum(-1, keepdim=True)
        shape = s["idx"].shape
        return {"idx": idx.to(torch.int32).view(shape), "gate": (chosen * c["scale"]).view(shape)}
    idx, d = s["idx"].long().view(-1, k), s["d_gate"].to(torch.float64).view(-1, k) * c["scale"]
    p = torch.take_along_dim(score, idx, -1)
    grad = torch.zeros_like(score)
    if c["renorm"]:  # g_j = p_j / P: dg_j/dl_i = g_j (d log p_j - sum_m g_m d log p_m)
        g = p / p.sum(-1, keepdim=True)
        slope = (1.0 - p) if c["score"] == "sigmoid" else 1.0  # d log p / dl, the softmax's common part cancels
        grad.scatter_(-1, idx, g * (d - (d * g).sum(-1, keepdim=True)) * slope)
    elif c["score"] == "sigmoid":
        grad.scatter_(-1, idx, d * p * (1.0 - p))
    else:
        grad.scatter_(-1, idx, d * p)
        grad -= score * (d * p).sum(-1, keepdim=True)
    return grad.view(s["logits"].shape)


def _exact_norm(c, s):
    H, n = c["H"], c["R"] * c["T"]
    f = torch.float64
    rows = {name: s[name].view(n, H) for name in ("x", "residual", "d_y", "d_residual_out") if name in s}
    rank = torch.arange(n, device="cuda") // c["T"]
    w = s["weight"].to(f)
    w1 = s["post"].to(f) if c["post"] else None
    sums = {"d_weight": torch.zeros(H, dtype=f, device="cuda")}
    if c["gate"] == "channel":
        sums["d_gate"] = torch.zeros(H, dtype=f, device="cuda")
    elif c["gate"] == "rank":
        sums["d_gate"] = torch.zeros(c["R"], H, dtype=f, device="cuda")
    if c["post"]:
        sums["d_post"] = torch.zeros(H, dtype=f, device="cuda")
    parts = {}
    for a in range(0, n, CHUNK):
        b = min(n, a + CHUNK)
        x, res = rows["x"][a:b].to(f), rows["residual"][a:b].to(f)
        inv1 = 1.0 / torch.sqrt(x.square().sum(-1, keepdim=True) / H + EPS)
        u = x * inv1 * w1 if c["post"] else x
        if c["gate"] == "none":
            gate = torch.ones(1, H, dtype=f, device="cuda")
        elif c["gate"] == "channel":
            gate = s["g"].to(f).view(1, H)
        elif c["gate"] == "rank":
            gate = s["g"].to(f)[rank[a:b]]
        else:
            gate = s["g"].view(n, H)[a:b].to(f)
        z = res * c["alpha"] + gate * u * c["beta"]
        inv2 = 1.0 / torch.sqrt(z.square().sum(-1, keepdim=True) / H + EPS)
        if c["op"] == NORM:
            v = z * inv2 * w
            step = {"residual": z}
            if c["bits"] == 16:
                step["y"] = v
            else:
                peak = v.abs().amax(-1)
                step["q"], step["scale"] = v * LOW8 / peak.unsqueeze(-1), peak / LOW8
        else:
            dy, dro = rows["d_y"][a:b].to(f), rows["d_residual_out"][a:b].to(f)
            unit = z * inv2
            sums["d_weight"] += (dy * unit).sum(0)
            t = dy * w
            dz = dro + inv2 * (t - unit * ((t * unit).sum(-1, keepdim=True) / H))
            step = {"d_residual": dz * c["alpha"]}
            dbranch = dz * c["beta"]
            if c["gate"] == "channel":
                sums["d_gate"] += (dbranch * u).sum(0)
            elif c["gate"] == "rank":
                sums["d_gate"].index_add_(0, rank[a:b], dbranch * u)
            elif c["gate"] == "token":
                step["d_gate"] = dbranch * u
            du = dbranch * gate
            if c["post"]:
                unit = x * inv1
                sums["d_post"] += (du * unit).sum(0)
                t = du * w1
                du = inv1 * (t - unit * ((t * unit).sum(-1, keepdim=True) / H))
            step["d_x"] = du
        for name, t in step.items():
            parts.setdefault(name, []).append(t)
    out = {name: torch.cat(ts) for name, ts in parts.items()}
    lead = (c["R"], c["T"])
    out = {name: t.view(*lead, *t.shape[1:]) for name, t in out.items()}
    if c["op"] == NORM:
        return out
    out.update(sums)
    names = ["d_residual", "d_weight"] + (["d_gate"] if c["gate"] != "none" else []) + (["d_post"] if c["post"] else [])
    return {name: out[name] for name in names + ["d_x"]}


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] in (ROUTE, ROUTE_GRAD):
        return _exact_route(c, s)
    if c["op"] != COMBINE_GRAD:
        return _exact_norm(c, s)
    H, k = c["H"], c["k"]
    y, slot = s["y"], s["slot_map"].flatten().long()
    d_gate = torch.empty(slot.numel(), dtype=torch.float64, device="cuda")
    d_y = torch.empty(y.shape, dtype=torch.float64, device="cuda")
    gate, d_out = s["gate"].flatten().to(torch.float64), s["d_out"].view(-1, H)
    for a in range(0, slot.numel(), 8 * CHUNK):
        at = slot[a:a + 8 * CHUNK]
        token = torch.arange(a, a + at.numel(), device="cuda") // k
        d = d_out.index_select(0, token).to(torch.float64)
        d_gate[a:a + at.numel()] = torch.einsum("nh,nh->n", y.index_select(0, at).to(torch.float64), d)
        d_y.index_copy_(0, at, d.mul_(gate[a:a + at.numel()].unsqueeze(-1)))
    return {"d_y": d_y, "d_gate": d_gate.view(s["gate"].shape)}
