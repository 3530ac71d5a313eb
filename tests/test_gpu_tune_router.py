"""The operators together, as the examples use them: a block with norms around it and a router by scores, and
its gradient with frozen experts.

The gradients against those of the block in 64 bits, the choice held fixed.  On its way a value is rounded
to bf16 at most 8 times (y, the experts' inner and outer rows, and the same and the tokens on the way back), each
rounding 2^-8 of itself at most, so 2^-5 of a tensor's norm; the stages that take differences (the router's
gradient, the norms' projections) leave at least half of what they are given here, a factor of 2: 2^-4."""
import os
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

import combine_device_resident_gb300 as A  # noqa: E402
from tests.test_gpu_block_norm import reference  # noqa: E402
from tests.test_gpu_route_scores import choose, gates  # noqa: E402

DEV = torch.device("cuda", 0)
RULES = {"sigmoid groups": dict(score="sigmoid", groups=4, groups_kept=2, group_best=2, scale=2.5),
         "sigmoid": dict(score="sigmoid", renormalize=False),
         "softmax": dict(score="softmax", renormalize=False, scale=1.5),
         "softmax groups": dict(score="softmax", groups=4, groups_kept=3)}


def near(got, ref, tol=2.0 ** -4):
    off = ((got.double() - ref.double()).norm() / ref.double().norm()).item()
    assert off < tol, off


@pytest.mark.parametrize("form", ["bf16", "8bit", "4bit"])
def test_block_with_norms_around_it(form):
    from moe_block import MoeBlock

    rule = A.RouteRule(**RULES["sigmoid groups"])
    b = MoeBlock(4, 16, 19, 256, 192, 3, form, rule=rule, sandwich=True, residual_scale=0.75, branch_scale=0.5)
    g = torch.Generator(device=DEV).manual_seed(3)
    x, r = (torch.randn(b.R, b.T, b.H, generator=g, device=DEV).bfloat16() for _ in range(2))
    b.bias.copy_(torch.round(torch.randn(16, generator=g, device=DEV) * 30) * 1e-3)
    kept = r.clone()
    out = b(x, r).clone()
    f = reference(dict(x=x, residual=kept, post_weight=b.w_post, gate=b.block_gate), 0.75, 0.5)
    near(r, f["z"], 2.0 ** -8)
    near(b.y, f["z"] * f["r2"] * b.w_norm.double(), 2.0 ** -8)
    want = choose(b.logits, b.bias, rule, b.k)
    assert torch.equal(b.topk.cpu().long(), want)
    near(b.gate.cpu(), gates(b.logits, want, rule), 2.0 ** -18)
    parts = b.gate.double().unsqueeze(-1) * b.expert_out[b.slot_map.long()].double()
    near(out, parts.sum(2), 2.0 ** -8)
    # a replayed graph follows its inputs
    xin, rin = x.clone(), kept.clone()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        b(xin, rin)
    xin.copy_(x)
    rin.copy_(kept)
    b.out.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(b.out, out) and torch.equal(rin, r) and b.status() == 0
    b.close()


def reference_grads(t, x, residual, d_out, d_res):
    b = t.block
    leaves = {n: getattr(b, n).double().requires_grad_() for n in t.params}
    leaves["x"], leaves["residual"] = x.double().requires_grad_(), residual.double().requires_grad_()
    f = reference(dict(x=leaves["x"], residual=leaves["residual"], post_weight=leaves["w_post"], gate=leaves["block_gate"]),
                  b.residual_scale, b.branch_scale)
    y = f["z"] * f["r2"] * leaves["w_norm"]
    logits = y @ leaves["w_router"].T
    idx = b.topk.long()
    if b.rule.renormalize:
        base = torch.nn.functional.logsigmoid(logits) if b.rule.score else logits
        gate = torch.softmax(base.gather(-1, idx), -1) * b.rule.scale
    else:
        gate = (torch.sigmoid(logits) if b.rule.score else torch.softmax(logits, -1)).gather(-1, idx) * b.rule.scale
    out = torch.zeros_like(y)
    for j in range(b.k):
        pre = torch.einsum("rth,rtnh->rtn", y, b.w_in.double()[idx[..., j]])
        g, u = pre.chunk(2, dim=-1)
        expert = torch.einsum("rtf,rthf->rth", g * torch.sigmoid(g) * u, b.w_out.double()[idx[..., j]])
        out = out + gate[..., j:j + 1] * expert
    loss = (out * d_out.double()).sum() + (f["z"] * d_res.double()).sum()
    return dict(zip(leaves, torch.autograd.grad(loss, list(leaves.values()))))


@pytest.mark.parametrize("name", RULES)
def test_gradients_of_the_block(name):
    from tune_router import TunedBlock

    t = TunedBlock(2, 16, 21, 256, 128, 3, A.RouteRule(**RULES[name]), residual_scale=0.75, branch_scale=1.5)
    g = torch.Generator(device=DEV).manual_seed(5)
    x, r, d_out, d_res = (torch.randn(2, 21, 256, generator=g, device=DEV).bfloat16() for _ in range(4))
    t.forward(x, r)
    t.backward(x, r, d_out, d_res)
    want = reference_grads(t, x, r, d_out, d_res)
    for n, d in t.params.items():
        near(getattr(t, d), want[n])
    near(t.d_x, want["x"])
    near(t.d_residual, want["residual"])
    assert t.block.status() == 0
    t.close()


def test_forward_and_backward_captured():
    """One graph of both; replayed on other inputs it gives what eager calls give, bit for bit."""
    from tune_router import TunedBlock

    t = TunedBlock(4, 32, 33, 512, 128, 4, A.RouteRule(**RULES["sigmoid groups"]))
    g = torch.Generator(device=DEV).manual_seed(6)
    first, second = ([torch.randn(4, 33, 512, generator=g, device=DEV).bfloat16() for _ in range(4)] for _ in range(2))
    names = [*t.params.values(), "d_x", "d_residual", "d_logits"]

    def run(x, r, d_out, d_res):
        t.forward(x, r)
        t.backward(x, r, d_out, d_res)

    want = []
    for inputs in (first, second):
        run(*inputs)
        want.append([getattr(t, n).clone() for n in names])
    held = [i.clone() for i in first]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        run(*held)
    for inputs, grads in zip((first, second), want):
        for h, i in zip(held, inputs):
            h.copy_(i)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(getattr(t, n), w) for n, w in zip(names, grads))
    assert t.block.status() == 0
    t.close()


@pytest.mark.parametrize("example,args", [
    ("tune_router", ["--steps", "3", "--tokens", "16", "--hidden", "256", "--inner", "128"]),
    ("moe_block", ["--form", "bf16", "--sandwich", "--score", "sigmoid", "--groups", "4", "--groups-kept", "2", "--tokens", "8",
                   "--hidden", "512", "--inner", "128", "--steps", "2"])])
def test_examples_run(example, args, capsys):
    __import__(example).main(args)
    assert "status 0" in capsys.readouterr().out
