"""The example block: every stage against 64 bits from the values the stage before it left in memory, and a
captured block against an eager one."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

import combine_device_resident_gb300 as A  # noqa: E402
from tests.test_gpu_experts import BF, check_rows8, norm_ref, product_ref, within  # noqa: E402

DEV = torch.device("cuda", 0)


def make(form, **kw):
    from moe_block import MoeBlock

    args = dict(R=4, E=8, T=19, H=256, F=192, k=2)
    args.update(kw)
    b = MoeBlock(form=form, **args)
    g = torch.Generator(device=DEV).manual_seed(11)
    shape = (b.R, b.T, b.H)
    return b, torch.randn(shape, generator=g, device=DEV).bfloat16(), torch.randn(shape, generator=g, device=DEV).bfloat16()


def weights64(b, which):
    w, s = (b.w_in, b.s_in) if which == "in" else (b.w_out, b.s_out)
    if b.form == "bf16":
        return w.double()
    if b.form == "8bit":
        return w.double() * s.double().unsqueeze(-1)
    return A.unpack_weights_w4(w, s).double()


def rows64(t, form):
    if form != "8bit":
        return t.double()
    q, s = A.rows8_parts(t.view(torch.uint8))
    return q.double() * s.double().unsqueeze(-1)


@pytest.mark.parametrize("form", ["bf16", "8bit", "4bit"])
@pytest.mark.parametrize("k", [1, 3])
def test_every_stage(form, k):
    b, x, r = make(form, k=k)
    r0 = r.clone()
    out = b(x, r)
    torch.cuda.synchronize()
    assert b.status() == 0
    z, v = norm_ref(x, r0, b.w_norm, b.eps)
    within(r, z, z.abs() * (BF + 2.0 ** -23))
    within(b.y, v, v.abs() * (BF + 2.0 ** -18) + 1e-38)
    if form == "8bit":
        check_rows8(b.rows8, v, 2.0 ** -18)
    # the dispatch: every assignment's row is its token's, bit for bit
    sent = b.y if form != "8bit" else b.rows8.view(torch.bfloat16)
    slots = b.slot_map.long()
    assert sorted(slots.flatten().tolist()) == list(range(b.R * b.T * k))
    want = sent.unsqueeze(2).expand(-1, -1, k, -1)
    assert torch.equal(b.recv[slots.flatten()].view(torch.int16), want.reshape(-1, want.shape[-1]).view(torch.int16))
    # the experts, each row by its own
    expert = torch.empty(b.R * b.T * k, dtype=torch.long, device=DEV)
    expert[slots.flatten()] = b.topk.long().flatten()
    x1, w1, w2 = rows64(b.recv, form), weights64(b, "in"), weights64(b, "out")
    x2 = rows64(b.inner if form != "8bit" else b.inner8, form)
    if form == "8bit":
        check_rows8(b.inner8, b.inner.double(), 2.0 ** -22)
    for e in expert.unique().tolist():
        at = expert == e
        ref, tol = product_ref(None, x1[at], w1[e], None, True, b.H)
        within(b.inner[at], ref, tol)
        ref, tol = product_ref(None, x2[at], w2[e], None, False, b.F)
        within(b.expert_out[at], ref, tol)
    # the combine: k products and sums in fp32, then bf16
    parts = b.gate.double().unsqueeze(-1) * b.expert_out[slots].double()
    ref = parts.sum(2)
    within(out, ref, ref.abs() * BF + parts.abs().sum(2) * k * 2.0 ** -23)
    b.close()


@pytest.mark.parametrize("form", ["bf16", "8bit", "4bit"])
def test_captured_block_follows_its_inputs(form):
    b, x, r = make(form)
    x2, r2 = x.flip(1).contiguous() * 2, r.flip(0).contiguous()
    want = []
    for xs, rs in ((x, r), (x2, r2)):
        rs = rs.clone()
        want.append((b(xs, rs).clone(), rs))
    xin, rin = x.clone(), r.clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        b(xin, rin)
    for (xs, rs), (out, res) in zip(((x, r), (x2, r2)), want):
        xin.copy_(xs)
        rin.copy_(rs)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(b.out.view(torch.int16), out.view(torch.int16))
        assert torch.equal(rin.view(torch.int16), res.view(torch.int16))
    assert b.status() == 0
    b.close()


@pytest.mark.parametrize("form", ["bf16", "8bit", "4bit"])
def test_one_token(form):
    b, x, r = make(form, R=1, E=4, T=1, k=1)
    out = b(x, r)
    torch.cuda.synchronize()
    assert b.status() == 0 and torch.isfinite(out.float()).all() and out.float().abs().max() > 0
    b.close()
