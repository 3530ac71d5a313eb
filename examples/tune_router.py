"""Tuning what stands around frozen experts: the router, the norms and the block's gate.

One MoE block forward (``moe_block.MoeBlock`` with norms around it and a router by scores), its gradient,
and a step:

    d_out -> combine_grad -> d_expert_out, d_gate
    d_gate -> route_scores_grad -> d_logits -> the router's weights, and its input
    d_expert_out -> the experts' products with their weights turned over -> combine with gates of one
                    (the dispatch's gradient) -> the tokens
    tokens -> block_norm_grad -> the block before, the residual stream, the norms' weights, the gate

The bias of the choice has no gradient: it is moved by the experts' loads, up for those with fewer rows
than the mean.  Counts, gradients and weights stay on the GPU, so forward and backward are one CUDA graph.

Run it:  python examples/tune_router.py --ranks 4 --experts 32 --tokens 128 --steps 20
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
sys.path.insert(0, HERE)
sys.path.insert(0, os.path.dirname(HERE))

import combine_device_resident_gb300 as a2av  # noqa: E402
from moe_block import MoeBlock  # noqa: E402


class TunedBlock:
    """A block with frozen bf16 experts and the gradients of the rest.

    ``params``: the names of the tuned weights and their gradients, both attributes: fp32 ``d_router`` [E][H],
    ``d_norm``, ``d_post`` and ``d_block_gate`` [H]; ``d_x`` and ``d_residual`` go on to the block before."""

    params = {"w_router": "d_router", "w_norm": "d_norm", "w_post": "d_post", "block_gate": "d_block_gate"}

    def __init__(self, R, E, T, H, F, k, rule, device="cuda:0", seed=0, residual_scale=1.0, branch_scale=1.0):
        self.block = b = MoeBlock(R, E, T, H, F, k, device=device, seed=seed, rule=rule, sandwich=True,
                                  residual_scale=residual_scale, branch_scale=branch_scale)
        dev = b.out.device
        self.w_in_t = b.w_in.transpose(1, 2).contiguous()     # [E][H][2F]: laid out once, the experts are frozen
        self.w_out_t = b.w_out.transpose(1, 2).contiguous()   # [E][F][H]
        bf, f32 = dict(dtype=torch.bfloat16, device=dev), dict(dtype=torch.float32, device=dev)
        arena, tokens = b.plan.arena_rows, (R, T, H)
        self.residual_out = torch.empty(tokens, **bf)
        self.d_expert_out, self.d_recv = torch.empty(arena, H, **bf), torch.empty(arena, H, **bf)
        self.pre, self.d_pre = torch.empty(arena, 2 * F, **bf), torch.empty(arena, 2 * F, **bf)
        self.d_inner = torch.empty(arena, F, **bf)
        self.d_gate, self.ones = torch.empty(R, T, k, **f32), torch.ones(R, T, k, **f32)
        self.d_logits = torch.empty(R, T, E, **f32)
        self.d_y, self.d_x, self.d_residual = (torch.empty(tokens, **bf) for _ in range(3))
        self.d_router = torch.empty(E, H, **f32)
        self.d_norm, self.d_post, self.d_block_gate = (torch.empty(H, **f32) for _ in range(3))
        self.scratch = b.plan.new_norm_scratch()

    def forward(self, x, residual):
        return self.block(x, residual, self.residual_out)

    def backward(self, x, residual, d_out, d_residual_out):
        """Gradients for the inputs of the last ``forward``, from those of its output and of ``residual_out``."""
        b, p = self.block, self.block.plan
        p.combine_grad(d_out, b.expert_out, b.gate, b.slot_map, d_y=self.d_expert_out, d_gate=self.d_gate)
        # the experts: every row of the packed windows is live, as every token takes part
        p.expert_matmul(self.d_expert_out, self.w_out_t, b.splits, self.d_inner)
        p.expert_matmul(b.recv, b.w_in, b.splits, self.pre)
        g, u, d = (t.float() for t in (*self.pre.chunk(2, dim=-1), self.d_inner))
        s = torch.sigmoid(g)
        self.d_pre[:, :b.F] = d * u * s * (1.0 + g * (1.0 - s))
        self.d_pre[:, b.F:] = d * g * s
        p.expert_matmul(self.d_pre, self.w_in_t, b.splits, self.d_recv)
        p.combine(self.d_recv, self.ones, b.slot_map, self.d_y)
        # the router: its projection is a library product, as in the block
        p.route_scores_grad(b.logits, b.topk, self.d_gate, self.d_logits, b.rule)
        d_logits = self.d_logits.view(-1, b.E)
        torch.mm(d_logits.T, b.y32, out=self.d_router)
        self.d_y += torch.mm(d_logits, b.router32.T).view_as(self.d_y)
        p.block_norm_grad(x, residual, self.d_x, self.d_residual, weight=b.w_norm, d_y=self.d_y,
                          d_residual_out=d_residual_out, post_weight=b.w_post, gate=b.block_gate, d_weight=self.d_norm,
                          d_post_weight=self.d_post, d_gate=self.d_block_gate, scratch=self.scratch,
                          residual_scale=b.residual_scale, branch_scale=b.branch_scale, eps=b.eps)

    def step(self, rate, bias_rate):
        """A step down the gradients, and the bias after the loads."""
        b = self.block
        for name, grad in self.params.items():
            w = getattr(b, name)
            w.copy_(w.float() - rate * getattr(self, grad))
        b.router32.copy_(b.w_router.float().T)
        load = b.splits.send_counts.sum(0).float()
        b.bias += bias_rate * torch.sign(load.mean() - load)

    def close(self):
        self.block.close()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--ranks", type=int, default=4)
    ap.add_argument("--experts", type=int, default=32)
    ap.add_argument("--tokens", type=int, default=128, help="per rank")
    ap.add_argument("--hidden", type=int, default=1024)
    ap.add_argument("--inner", type=int, default=512)
    ap.add_argument("--topk", type=int, default=4)
    ap.add_argument("--score", choices=["softmax", "sigmoid"], default="sigmoid")
    ap.add_argument("--groups", type=int, default=4)
    ap.add_argument("--groups-kept", type=int, default=2)
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--rate", type=float, default=1e-3)
    ap.add_argument("--bias-rate", type=float, default=1e-3)
    a = ap.parse_args(argv)
    rule = a2av.RouteRule(score=a.score, groups=a.groups, groups_kept=a.groups_kept, group_best=2)
    tuned = TunedBlock(a.ranks, a.experts, a.tokens, a.hidden, a.inner, a.topk, rule)
    dev = tuned.block.out.device
    shape = (a.ranks, a.tokens, a.hidden)
    x, residual, target = (torch.randn(shape, device=dev).to(torch.bfloat16) for _ in range(3))
    d_residual_out = torch.zeros_like(x)
    for i in range(a.steps):
        out = tuned.forward(x, residual)
        diff = out.float() - target.float()
        tuned.backward(x, residual, diff.to(torch.bfloat16), d_residual_out)
        tuned.step(a.rate, a.bias_rate)
        if i % 5 == 0 or i == a.steps - 1:
            load = tuned.block.splits.send_counts.sum(0)
            print(f"step {i}: loss {0.5 * diff.square().sum(-1).mean().item():.4f}, rows per expert "
                  f"{load.min().item()}..{load.max().item()}")
    print(f"status {tuned.block.status()}")
    tuned.close()


if __name__ == "__main__":
    main()
