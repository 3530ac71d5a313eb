"""One MoE block on the library's kernels, from the residual stream to the residual stream.

    norm (+ residual)  ->  router  ->  dispatch  ->  experts (SwiGLU, down)  ->  combine

Routing stays on the GPU, nothing is padded and nothing synchronises, so the block is one CUDA
graph.  Three forms of the experts:

    bf16   bf16 rows and weights
    8bit   the norm writes 8-bit rows with their scales, the dispatch moves those (half the
           bytes), both products are e4m3
    4bit   bf16 rows, 4-bit weights with group scales: for decode

Run it:  python examples/moe_block.py --form 8bit --ranks 8 --experts 16 --tokens 64
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import combine_device_resident_gb300 as a2av  # noqa: E402
from combine_device_resident_gb300.binding import ROW8_TAIL  # noqa: E402

FORMS = ("bf16", "8bit", "4bit")


class MoeBlock:
    """R emulated ranks of T tokens, hidden H, E experts of inner width F, top-k.

    Weights are random; ``w_norm`` [H], ``w_router`` [E][H], gate and up ``w_in`` [E][2F][H], ``w_out`` [E][H][F].
    All buffers are made here; ``__call__`` only enqueues kernels on the current stream."""

    def __init__(self, R, E, T, H, F, k, form="bf16", group=64, device="cuda:0", seed=0):
        if form not in FORMS:
            raise ValueError(f"form must be one of {FORMS}, got {form!r}")
        self.form, self.eps = form, 1e-6
        self.R, self.E, self.T, self.H, self.F, self.k = R, E, T, H, F, k
        dev = torch.device(device)
        g = torch.Generator(device=dev).manual_seed(seed)

        def normal(*shape, std=1.0):
            return torch.randn(shape, generator=g, device=dev).mul_(std)

        self.w_norm = (1.0 + normal(H, std=0.1)).to(torch.bfloat16)
        self.w_router = normal(E, H, std=H ** -0.5).to(torch.bfloat16)
        self.router32 = self.w_router.float().T             # what its product takes, laid out once
        w_in, w_out = normal(E, 2 * F, H, std=H ** -0.5), normal(E, H, F, std=F ** -0.5)
        self.s_in = self.s_out = None
        if form == "bf16":
            self.w_in, self.w_out = w_in.to(torch.bfloat16), w_out.to(torch.bfloat16)
        elif form == "8bit":
            (self.w_in, self.s_in), (self.w_out, self.s_out) = map(a2av.quantize_weights, (w_in, w_out))
        else:
            (self.w_in, self.s_in), (self.w_out, self.s_out) = (a2av.pack_weights_w4(w, group) for w in (w_in, w_out))

        # The plan of the tokens: norm, router, experts, combine.  8-bit rows travel through a plan of
        # their own length: a row of H + 16 bytes moves like a bf16 row of (H + 16) / 2.
        self.plan = a2av.Plan(R, E, T, H, k, device=dev, recv_order="expert")
        self.rows_plan = self.plan
        if form == "8bit":
            self.rows_plan = a2av.Plan(R, E, T, (H + ROW8_TAIL) // 2, k, device=dev, recv_order="expert")
        self.splits = self.plan.new_splits()
        arena = self.plan.arena_rows
        bf = dict(dtype=torch.bfloat16, device=dev)
        self.y = torch.empty(R, T, H, **bf)                 # normed tokens: the router reads them, and the bf16 experts
        self.y32 = torch.empty(R * T, H, dtype=torch.float32, device=dev)  # the same for the router's product
        self.rows8 = self.plan.new_rows8((R, T), H) if form == "8bit" else None
        self.logits = torch.empty(R, T, E, dtype=torch.float32, device=dev)
        self.topk = torch.empty(R, T, k, dtype=torch.int32, device=dev)
        self.gate = torch.empty(R, T, k, dtype=torch.float32, device=dev)
        self.recv = torch.empty(arena, self.rows_plan.H, **bf)
        self.slot_map = torch.empty(R, T, k, dtype=torch.int32, device=dev)
        self.out = torch.empty(R, T, H, **bf)
        self.inner = torch.empty(arena, F, **bf)
        self.inner8 = self.plan.new_rows8(arena, F) if form == "8bit" else None
        self.expert_out = torch.empty(arena, H, **bf)

    def __call__(self, x, residual):
        """The experts' weighted output for x + residual, normed; the sum goes into ``residual`` (the next
        block's residual stream)."""
        p, rows = self.plan, self.rows_plan
        p.rms_norm(x, self.w_norm, y=self.y, rows8=self.rows8, residual=residual, residual_out=residual, eps=self.eps)
        self.y32.copy_(self.y.view(-1, self.H))
        torch.mm(self.y32, self.router32, out=self.logits.view(-1, self.E))  # the router's projection, a library product
        p.route(self.logits, self.topk, self.gate)
        sent = self.y if self.form != "8bit" else self.rows8.view(torch.bfloat16)
        rows.dispatch(sent, self.topk, self.splits, self.recv, self.slot_map)
        if self.form == "bf16":
            p.expert_matmul(self.recv, self.w_in, self.splits, self.inner, activation="swiglu")
            p.expert_matmul(self.inner, self.w_out, self.splits, self.expert_out)
        elif self.form == "8bit":
            p.expert_matmul(self.recv.view(torch.uint8), self.w_in, self.splits, self.inner, w_scale=self.s_in,
                            activation="swiglu")
            p.quantize_rows(self.inner, self.splits, self.inner8)
            p.expert_matmul(self.inner8, self.w_out, self.splits, self.expert_out, w_scale=self.s_out)
        else:
            p.expert_matmul_w4(self.recv, self.w_in, self.s_in, self.splits, self.inner, activation="swiglu")
            p.expert_matmul_w4(self.inner, self.w_out, self.s_out, self.splits, self.expert_out)
        p.combine(self.expert_out, self.gate, self.slot_map, self.out)
        return self.out

    def status(self):
        """Device status bits of both plans."""
        return self.plan.read_status() | self.rows_plan.read_status()

    def close(self):
        if self.rows_plan is not self.plan:
            self.rows_plan.close()
        self.plan.close()


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--form", choices=FORMS, default="8bit")
    ap.add_argument("--ranks", type=int, default=8)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--tokens", type=int, default=64, help="per rank")
    ap.add_argument("--hidden", type=int, default=5120)
    ap.add_argument("--inner", type=int, default=2048, help="an expert's inner width")
    ap.add_argument("--topk", type=int, default=2)
    ap.add_argument("--steps", type=int, default=50)
    a = ap.parse_args(argv)
    block = MoeBlock(a.ranks, a.experts, a.tokens, a.hidden, a.inner, a.topk, a.form)
    dev = block.out.device
    x = torch.randn(a.ranks, a.tokens, a.hidden, device=dev).to(torch.bfloat16)
    residual = torch.randn_like(x)
    for _ in range(3):
        block(x, residual)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        block(x, residual)
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    graph.replay()
    torch.cuda.synchronize()
    begin.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    tokens = a.ranks * a.tokens
    us = begin.elapsed_time(end) * 1e3 / a.steps
    rows = block.splits.recv_total.cpu().tolist()
    print(f"{a.form}: {tokens} tokens, {a.experts} experts, top-{a.topk}: {us:.1f} us a block, "
          f"{tokens / us:.2f} tokens/us; rows per rank {min(rows)}..{max(rows)}; status {block.status()}")
    block.close()


if __name__ == "__main__":
    main()
