"""Cases of the operators around the dispatch and the combine: the norm in front
(root-mean-square norm with the residual's addition, in bf16 or as 8-bit rows with
scales), the experts' products on the dispatched rows (bf16 or 8 bits, with or
without the SwiGLU), and the same with 4-bit weights for few rows.

A case is one call on the shapes of an MoE block: R ranks of T tokens, E experts,
top-k, hidden H; F is an expert's inner width.  The rows of the products lie as the
expert-grouped dispatch leaves them (packed windows), their sizes in the split arrays.
"""
import functools
import math

import torch

own = False

LOW8 = 448.0          # largest finite e4m3 value
SHIFTS = (0, 16, 4, 20, 8, 24, 12, 28)  # bit of k = 0..7 in a word of eight 4-bit weights
NORM, QUANT, MATMUL, MATMUL8, MATMUL4 = "norm", "quantize", "matmul", "matmul8", "matmul4"


def listed():
    return [
        # one decode step, a token per rank: the norm before an 8-bit dispatch; latency counts
        dict(name="norm 8x5120 to 8 bits", op=NORM, R=8, T=1, H=5120, bits=8),
        # a decode batch of 256 tokens per rank, bf16 rows
        dict(name="norm 2048x5120 bf16", op=NORM, R=8, T=256, H=5120, bits=16),
        # the prefill batch of the largest workload
        dict(name="norm 65536x7168 to 8 bits", op=NORM, R=32, T=2048, H=7168, bits=8),
        # the norm's 8-bit rows without the norm: the SwiGLU's output before the second 8-bit product
        dict(name="quantize 32768x2048", op=QUANT, R=16, E=128, T=1024, k=2, K=2048, routing="zipf", s=1.0),
        # decode, a token per rank: up to eight experts with a row or two each
        dict(name="matmul 8 rows swiglu", op=MATMUL, R=8, E=128, T=1, k=1, K=5120, N=2048, swiglu=True,
             routing="zipf", s=1.2),
        # an odd batch and an odd width, second product: ragged groups near 510 rows
        dict(name="matmul 8168 rows odd", op=MATMUL, R=8, E=16, T=1021, k=1, K=1416, N=5120, swiglu=False,
             routing="uniform", s=0.0),
        # prefill, top-2 with Zipf loads from a handful of rows to thousands
        dict(name="matmul 32768 rows swiglu", op=MATMUL, R=16, E=128, T=1024, k=2, K=5120, N=2048, swiglu=True,
             routing="zipf", s=1.0),
        # a decode batch in 8 bits: most experts have a few rows
        dict(name="matmul8 2048 rows swiglu", op=MATMUL8, R=8, E=128, T=256, k=1, K=5120, N=2048, swiglu=True,
             routing="zipf", s=1.2),
        # prefill in 8 bits, top-8 with a hot expert: the largest
        dict(name="matmul8 131072 rows swiglu", op=MATMUL8, R=32, E=256, T=512, k=8, K=7168, N=2048, swiglu=True,
             routing="hot", s=1.1),
        # one token, one expert, 4-bit weights
        dict(name="matmul4 1 row swiglu", op=MATMUL4, R=1, E=16, T=1, k=1, K=5120, N=2048, group=128, swiglu=True,
             routing="uniform", s=0.0),
        # second product of a small batch, fine groups
        dict(name="matmul4 64 rows", op=MATMUL4, R=8, E=128, T=4, k=2, K=2048, N=5120, group=32, swiglu=False,
             routing="zipf", s=1.0),
        # a decode batch over most of 256 experts
        dict(name="matmul4 1024 rows swiglu", op=MATMUL4, R=32, E=256, T=4, k=8, K=7168, N=2048, group=128,
             swiglu=True, routing="hot", s=1.1),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi, step):
    return max(step, _log(rng, lo, hi) // step * step)


def draw(rng):
    op = rng.choice([NORM, NORM, QUANT, MATMUL, MATMUL, MATMUL8, MATMUL8, MATMUL4, MATMUL4])
    R = rng.choice([1, 2, 4, 8, 16, 32])
    if op == NORM:
        return dict(op=op, R=R, T=_log(rng, 1, 65536 // R), H=_width(rng, 256, 7168, 16), bits=rng.choice([8, 16]))
    E = R * rng.choice([1, 2, 4, 8])
    k = min(E, rng.choice([1, 2, 4, 8]))
    routing = rng.choice(["uniform", "zipf", "zipf", "hot"])
    c = dict(op=op, R=R, E=E, T=1, k=k, routing=routing, s=round(rng.uniform(0.8, 1.3), 2))
    if op == QUANT:
        return dict(c, T=_log(rng, 1, max(1, 32768 // (R * k))), K=_width(rng, 64, 4096, 16))
    swiglu = rng.random() < 0.5
    wide, narrow = (256, 7168), (64, 2048)  # hidden widths, experts' inner widths
    if op == MATMUL4:
        group = rng.choice([32, 64, 128])
        return dict(c, T=_log(rng, 1, max(1, 1024 // (R * k))), K=_width(rng, *(wide if swiglu else narrow), group),
                    N=_width(rng, *(narrow if swiglu else wide), 8), group=group, swiglu=swiglu)
    step = 16 if op == MATMUL8 else 8
    return dict(c, T=_log(rng, 1, max(1, 32768 // (R * k))), K=_width(rng, *(wide if swiglu else narrow), step),
                N=_width(rng, *(narrow if swiglu else wide), 8), swiglu=swiglu)


# ---- inputs -------------------------------------------------------------------

def _routing(c, g):
    """Expert ids [R][T][k]: k draws without replacement from the case's law (the k largest of
    log p + Gumbel noise), the experts' order shuffled."""
    E, shape = c["E"], (c["R"], c["T"], c["E"])
    p = torch.arange(1, E + 1, dtype=torch.float64, device="cuda") ** -(0.0 if c["routing"] == "uniform" else c["s"])
    p = (p / p.sum())[torch.randperm(E, generator=g, device="cuda")]
    if c["routing"] == "hot" and E > 1:  # expert 0 takes three tenths of the draws
        p[0] = 0.0
        p = p * (0.7 / p.sum())
        p[0] = 0.3
    u = torch.rand(shape, generator=g, device="cuda", dtype=torch.float64).clamp_(1e-300, 1.0 - 1e-16)
    return torch.topk(torch.log(p) - torch.log(-torch.log(u)), c["k"], dim=-1).indices


def _layout(c, g):
    """The split arrays of the expert-grouped receive order, packed windows, and the same as
    (expert, first row, end) of the experts that have rows."""
    R, E, epr = c["R"], c["E"], c["E"] // c["R"]
    idx = _routing(c, g)
    src = torch.arange(R, device="cuda").view(R, 1, 1)
    counts = torch.bincount((src * E + idx).flatten(), minlength=R * E).view(R, R, epr)  # [source][d][le]
    per = counts.permute(1, 2, 0).contiguous()                                            # [d][le][source]
    first = (per.view(R, -1).cumsum(1) - per.view(R, -1)).view(R, epr, R)
    total = per.view(R, -1).sum(1)
    a = {"recv_expert_counts": counts.permute(1, 0, 2), "recv_expert_offsets": first.permute(0, 2, 1),
         "recv_total": total, "window_base": total.cumsum(0) - total}
    a = {n: t.to(torch.int32).contiguous() for n, t in a.items()}
    rows = per.sum(2).flatten().tolist()
    ends = torch.tensor(rows).cumsum(0).tolist()
    return a, [(e, b - n, b) for e, (n, b) in enumerate(zip(rows, ends)) if n]


def _to8(v):
    """fp32 rows as (e4m3, scale): scale = max|v| / 448."""
    a = v.abs().amax(-1)
    return (v * (LOW8 / a).unsqueeze(-1)).clamp_(-LOW8, LOW8).to(torch.float8_e4m3fn), a / LOW8


def _rows8(lead, K):
    """8-bit rows as the framework keeps them: K bytes of e4m3, the fp32 scale, padding to 16 bytes; and
    views of the values and of the scales."""
    rows8 = torch.zeros(*lead, K + 16, dtype=torch.uint8, device="cuda")
    return rows8, rows8[..., :K].view(torch.float8_e4m3fn), rows8[..., K:K + 4].view(torch.float32)[..., 0]


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)

    s = {"case": c}
    if c["op"] == NORM:
        shape = (c["R"], c["T"], c["H"])
        # a residual stream some layers deep, and what the attention adds to it; a norm's weights lie near 1
        s["x"] = normal(*shape).to(torch.bfloat16)
        s["residual"] = normal(*shape).mul_(3.0).to(torch.bfloat16)
        s["weight"] = normal(c["H"]).mul_(0.1).add_(1.0).to(torch.bfloat16)
        s["residual_out"] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        if c["bits"] == 8:
            s["rows8"], s["q"], s["scale"] = _rows8(shape[:2], c["H"])
        else:
            s["y"] = torch.zeros(shape, dtype=torch.bfloat16, device="cuda")
        return s
    s["splits"], s["segments"] = _layout(c, g)
    M, K = c["R"] * c["T"] * c["k"], c["K"]
    x = normal(M, K)
    if c["op"] == QUANT or not c["swiglu"]:  # what a SwiGLU gives
        x = x * torch.sigmoid(x) * normal(M, K)
    if c["op"] == QUANT:
        s["x"] = x.to(torch.bfloat16)
        s["rows8"], s["q"], s["scale"] = _rows8((M,), K)
        return s
    if c["op"] == MATMUL8:
        s["x"], q, scale = _rows8((M,), K)
        v, a = _to8(x)
        q.copy_(v)
        scale.copy_(a)
    else:
        s["x"] = x.to(torch.bfloat16)
    del x
    wide = c["N"] * (2 if c["swiglu"] else 1)
    if c["op"] == MATMUL:
        s["w"] = torch.empty(c["E"], wide, K, dtype=torch.bfloat16, device="cuda")
        for e in range(c["E"]):
            s["w"][e] = normal(wide, K).mul_(K ** -0.5)
    elif c["op"] == MATMUL8:
        s["w"] = torch.empty(c["E"], wide, K, dtype=torch.float8_e4m3fn, device="cuda")
        s["w_scale"] = torch.empty(c["E"], wide, dtype=torch.float32, device="cuda")
        for e in range(c["E"]):
            s["w"][e], s["w_scale"][e] = _to8(normal(wide, K).mul_(K ** -0.5))
    else:
        # eight 4-bit weights a word; their scales such that the weights' spread is that of the others
        s["w"] = torch.randint(-2 ** 31, 2 ** 31, (c["E"], wide, K // 8), generator=g, device="cuda",
                               dtype=torch.int64).to(torch.int32)
        s["w_scale"] = (normal(c["E"], wide, K // c["group"]).abs_().add_(0.5).mul_(0.2 * K ** -0.5)).to(torch.bfloat16)
    s["y"] = torch.zeros(M, c["N"], dtype=torch.bfloat16, device="cuda")
    return s


# ---- the plain forms ----------------------------------------------------------

def _swiglu(p):
    g, u = p.chunk(2, dim=-1)
    return g * torch.sigmoid(g) * u


def _weights(s, e, dtype):
    """Expert e's weights [rows][K] in `dtype`."""
    c = s["case"]
    if c["op"] == MATMUL:
        return s["w"][e].to(dtype)
    if c["op"] == MATMUL8:
        return s["w"][e].to(dtype) * s["w_scale"][e].to(dtype)[:, None]
    q = (s["w"][e][..., None] >> torch.tensor(SHIFTS, dtype=torch.int32, device="cuda")) & 15
    q = (q - 8).view(q.shape[0], -1, c["group"]).to(dtype)
    return (q * s["w_scale"][e].to(dtype)[..., None]).view(q.shape[0], -1)


def _product(s, e, a, b):
    c = s["case"]
    if c["op"] == MATMUL8:
        x = s["x"][a:b, :c["K"]].view(torch.float8_e4m3fn).float()
        x = x * s["x"][a:b, c["K"]:c["K"] + 4].view(torch.float32)
    else:
        x = s["x"][a:b].float()
    p = x @ _weights(s, e, torch.float32).T
    return (_swiglu(p) if c["swiglu"] else p).to(torch.bfloat16)


def _plain(s):
    c = s["case"]
    if c["op"] == NORM:
        z = s["x"].float() + s["residual"].float()
        v = z * torch.rsqrt((z * z).mean(-1, keepdim=True) + 1e-6) * s["weight"].float()
        out = {"residual": z.to(torch.bfloat16)}
        if c["bits"] == 16:
            return dict(out, y=v.to(torch.bfloat16))
        q, scale = _to8(v)
        return dict(out, q=q, scale=scale)
    if c["op"] == QUANT:
        q, scale = _to8(s["x"].float())
        return {"q": q, "scale": scale}
    return torch.cat([_product(s, e, a, b) for e, a, b in s["segments"]])


# ---- the framework's calls ----------------------------------------------------

@functools.lru_cache(maxsize=None)
def _plan(R, E, T, H, k):
    import combine_device_resident_gb300 as a2av

    return a2av.Plan(R, E, T, H, k, device="cuda:0", recv_order="expert")


def _handles(s):
    """The plan of the case's sizes and the dispatch's splits, as a program keeps them."""
    if "handles" not in s:
        c = s["case"]
        plan = _plan(c["R"], c.get("E", c["R"]), c["T"], c.get("H", c.get("K")), c.get("k", 1))
        splits = plan.new_splits()
        for name, t in s.get("splits", {}).items():
            getattr(splits, name).copy_(t)
        s["handles"] = plan, splits
    return s["handles"]


def _own(s):
    plan, splits = _handles(s)
    c = s["case"]
    if c["op"] == NORM:
        plan.rms_norm(s["x"], s["weight"], residual=s["residual"], residual_out=s["residual_out"], y=s.get("y"),
                      rows8=s.get("rows8"), eps=1e-6)
        out = {"residual": s["residual_out"]}
        return dict(out, y=s["y"]) if c["bits"] == 16 else dict(out, q=s["q"], scale=s["scale"])
    if c["op"] == QUANT:
        plan.quantize_rows(s["x"], splits, s["rows8"])
        return {"q": s["q"], "scale": s["scale"]}
    act = "swiglu" if c["swiglu"] else None
    if c["op"] == MATMUL4:
        plan.expert_matmul_w4(s["x"], s["w"], s["w_scale"], splits, s["y"], activation=act)
    else:
        plan.expert_matmul(s["x"], s["w"], splits, s["y"], w_scale=s.get("w_scale"), activation=act)
    return s["y"]


def run(s):
    return _own(s) if own else _plain(s)


# ---- what a pass cannot do without ---------------------------------------------

def _live(c):
    """Experts that have rows, in expectation (the routing is the seed's): each of E misses all
    R*T*k assignments with the probability its law gives."""
    p = [(i + 1) ** -(0.0 if c["routing"] == "uniform" else c["s"]) for i in range(c["E"])]
    p = [v / sum(p) for v in p]
    if c["routing"] == "hot" and c["E"] > 1:
        p = [0.3] + [v * 0.7 / sum(p[1:]) for v in p[1:]]
    return sum(1.0 - (1.0 - min(v, 1.0)) ** (c["R"] * c["T"] * c["k"]) for v in p)


def work(c):
    if c["op"] == NORM:
        n = c["R"] * c["T"]
        out = c["H"] + 4 if c["bits"] == 8 else 2 * c["H"]
        return {"bytes": n * (6 * c["H"] + out) + 2 * c["H"], "flops": 6 * n * c["H"]}
    M, K = c["R"] * c["T"] * c["k"], c["K"]
    if c["op"] == QUANT:
        return {"bytes": M * (3 * K + 4), "flops": 2 * M * K}
    wide = c["N"] * (2 if c["swiglu"] else 1)
    weight = {MATMUL: 2.0 * K, MATMUL8: K + 4.0}.get(c["op"]) or K / 2 + 2.0 * K / c["group"]
    row = K + 4 if c["op"] == MATMUL8 else 2 * K
    return {"bytes": M * (row + 2 * c["N"]) + _live(c) * wide * weight, "flops": 2.0 * M * K * wide}


# ---- the definition in 64 bits --------------------------------------------------

def exact(c, seed):
    s = prepare(c, seed)
    d = torch.float64
    if c["op"] == NORM:
        z = s["x"].to(d).add_(s["residual"].to(d))
        v = z / (z.square().sum(-1, keepdim=True) / c["H"] + 1e-6).sqrt()
        v *= s["weight"].to(d)
        if c["bits"] == 16:
            return {"residual": z, "y": v}
        peak = v.abs().amax(-1)
        return {"residual": z, "q": v.mul_(448.0).div_(peak.unsqueeze(-1)), "scale": peak / 448.0}
    if c["op"] == QUANT:
        v = s["x"].to(d)
        peak = v.abs().amax(-1)
        return {"q": v * 448.0 / peak.unsqueeze(-1), "scale": peak / 448.0}
    K, N = c["K"], c["N"]
    if c["op"] == MATMUL8:
        x = s["x"][:, :K].view(torch.float8_e4m3fn).to(d) * s["x"][:, K:K + 4].view(torch.float32).to(d)
    else:
        x = s["x"].to(d)
    y = torch.zeros(x.shape[0], N, dtype=d, device="cuda")
    for e, a, b in s["segments"]:
        w = s["w"][e]
        if c["op"] == MATMUL4:
            full = torch.empty(w.shape[0], K, dtype=d, device="cuda")
            for i in range(8):  # k = 0, 2, 4, 6 from the low half of a word, 1, 3, 5, 7 from the high half
                full[:, i::8] = torch.bitwise_and(w >> (4 * (i // 2) + 16 * (i % 2)), 15).to(d) - 8.0
            w = full * s["w_scale"][e].to(d).repeat_interleave(c["group"], dim=1)
        elif c["op"] == MATMUL8:
            w = w.to(d) * s["w_scale"][e].to(d).unsqueeze(1)
        else:
            w = w.to(d)
        if c["swiglu"]:
            gate = torch.matmul(x[a:b], w[:N].t())
            y[a:b] = gate / (1.0 + torch.exp(-gate)) * torch.matmul(x[a:b], w[N:].t())
        else:
            y[a:b] = torch.matmul(x[a:b], w.t())
    return y
