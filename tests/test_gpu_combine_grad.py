"""The combine's gradient against its definition in 64 bits.

d_y is one fp32 product, rounded: equal to the plain form's bits.  d_gate sums exact
products (two of 8 bits each) in fp32: a thread adds at most 32 per piece of the
row in turn, then a tree of 5, then the warps (16 at most) in turn and the pieces: with
P pieces at most (32 + 5 + P + 16) roundings of 2^-24 of the sum of magnitudes.
"""
import pytest
import torch

import combine_device_resident_gb300 as A

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)
CANARY = 7.0
BAD_SLOT = 1 << 2


def setup(R, E, T, H, k, seed=0, **kw):
    g = torch.Generator(device=DEV).manual_seed(seed)
    plan = A.Plan(R, E, T, H, k, device=DEV, **kw)
    idx = torch.rand(R, T, max(E, k), generator=g, device=DEV).argsort(-1)[..., :k].to(torch.int32) % E
    gate = torch.rand(R, T, k, generator=g, device=DEV)
    x = torch.randn(R, T, H, generator=g, device=DEV).bfloat16()
    d_out = torch.randn(R, T, H, generator=g, device=DEV).bfloat16()
    y = torch.randn(plan.arena_rows, H, generator=g, device=DEV).bfloat16()
    recv, slot_map, _ = plan.new_buffers()
    plan.dispatch(x, idx.contiguous(), plan.new_splits(), recv, slot_map)
    plan.read_status(clear=True)
    return plan, d_out, y, gate, slot_map


def check(plan, d_out, y, gate, slot_map, d_y, d_gate, live=None):
    """d_y and d_gate of the tokens in `live` (all); rows and gates of no token untouched."""
    R, T, H, k = plan.R, plan.T, plan.H, plan.k
    part = torch.ones(R, T, dtype=torch.bool, device=DEV) if live is None else live
    slots = torch.where(slot_map >= plan.arena_rows, -1, slot_map)
    used = (slots >= 0) & part.unsqueeze(-1)
    at = slots[used].long()
    if d_y is not None:
        rows = torch.full((plan.arena_rows, H), CANARY, device=DEV).bfloat16()
        t = part.new_ones(R, T, k).nonzero()[used.flatten()]
        rows[at] = (gate[used].unsqueeze(-1) * d_out[t[:, 0], t[:, 1]].float()).bfloat16()
        assert torch.equal(d_y, rows)
    if d_gate is not None:
        ref = torch.zeros(R, T, k, dtype=torch.float64, device=DEV)
        size = torch.zeros_like(ref)
        for j in range(k):
            yj = y[slots[..., j].clamp(min=0).long()].double()
            prod = yj * d_out.double() * (slots[..., j] >= 0).unsqueeze(-1)
            ref[..., j], size[..., j] = prod.sum(-1), prod.abs().sum(-1)
        pieces = (H + 16383) // 16384
        off = (d_gate.double() - ref).abs() - size * (53 + pieces) * 2.0 ** -24
        assert (off[part] <= 1e-37).all()
        assert (d_gate[~part] == CANARY).all()


SHAPES = [(1, 1, 1, 8, 1), (1, 2, 3, 16, 2), (2, 4, 17, 264, 2), (8, 16, 5, 1032, 1), (4, 8, 9, 5120, 2),
          (2, 32, 6, 7168, 8), (1, 4, 2, 16400, 2), (1, 2, 3, 40008, 1), (1, 40, 7, 136, 32), (2, 6, 33, 4096, 6),
          (4, 32, 200, 64, 8), (1, 8, 1, 7168, 8), (3, 6, 50, 1024, 3), (64, 64, 2, 24, 5)]


@pytest.mark.parametrize("R,E,T,H,k", SHAPES)
@pytest.mark.parametrize("form", ["both", "rows", "gates", "in place"])
def test_combine_grad(R, E, T, H, k, form):
    plan, d_out, y, gate, slot_map = setup(R, E, T, H, k, H + k)
    before = plan.launches
    d_y = torch.full_like(y, CANARY) if form in ("both", "rows") else None
    d_gate = torch.full_like(gate, CANARY) if form != "rows" else None
    if form == "in place":
        was = y.clone()
        plan.combine_grad(d_out, y, gate, slot_map, d_y=y, d_gate=d_gate)
        y, d_y = was, y
    else:
        plan.combine_grad(d_out, y if form != "rows" else None, gate if form != "gates" else None, slot_map, d_y=d_y,
                          d_gate=d_gate)
    check(plan, d_out, y, gate, slot_map, d_y, d_gate)
    assert plan.read_status() == 0 and plan.launches == before + 1
    plan.close()


def test_same_bits_every_time():
    plan, d_out, y, gate, slot_map = setup(4, 8, 33, 5120, 4)
    out = []
    for _ in range(2):
        d_y, d_gate = torch.full_like(y, CANARY), torch.full_like(gate, CANARY)
        plan.combine_grad(d_out, y, gate, slot_map, d_y=d_y, d_gate=d_gate)
        out.append((d_y, d_gate))
    assert torch.equal(out[0][0], out[1][0]) and torch.equal(out[0][1], out[1][1])
    plan.close()


@pytest.mark.parametrize("H", [64, 5120])
def test_dropped_and_bad_slots(H):
    """Windows too small drop rows (slot -1); a slot past the arena counts as dropped and is flagged."""
    plan, d_out, y, gate, slot_map = setup(2, 4, 20, H, 2, window_mode="fixed", window_rows=15)
    assert (slot_map < 0).any()
    d_y, d_gate = torch.full_like(y, CANARY), torch.full_like(gate, CANARY)
    plan.combine_grad(d_out, y, gate, slot_map, d_y=d_y, d_gate=d_gate)
    check(plan, d_out, y, gate, slot_map, d_y, d_gate)
    assert plan.read_status() == 0
    slot_map[1, 3, 1] = plan.arena_rows
    slot_map[0, 5] = 2 ** 31 - 1
    slot_map[0, 6] = -2 ** 31
    d_y.fill_(CANARY)
    plan.combine_grad(d_out, y, gate, slot_map, d_y=d_y, d_gate=d_gate)
    check(plan, d_out, y, gate, slot_map, d_y, d_gate)
    assert plan.read_status() == BAD_SLOT
    plan.close()


@pytest.mark.parametrize("H", [64, 5120])
def test_tokens_that_take_no_part_are_left(H):
    R, T = 4, 6
    plan, d_out, y, gate, slot_map = setup(R, 8, T, H, 3)
    n = torch.tensor([0, 4, 9, -1], dtype=torch.int32, device=DEV)
    plan.set_active_tokens(n)
    live = torch.arange(T, device=DEV).view(1, T) < n.view(R, 1)
    d_y, d_gate = torch.full_like(y, CANARY), torch.full_like(gate, CANARY)
    plan.combine_grad(d_out, y, gate, slot_map, d_y=d_y, d_gate=d_gate)
    check(plan, d_out, y, gate, slot_map, d_y, d_gate, live)
    plan.close()


def test_special_values_stay_in_their_rows():
    plan, d_out, y, gate, slot_map = setup(1, 4, 9, 256, 2)
    d_out[0, 2, 3], gate[0, 4, 1], y[slot_map[0, 6, 0].long(), 5] = float("nan"), float("inf"), float("inf")
    d_y, d_gate = torch.full_like(y, CANARY), torch.full_like(gate, CANARY)
    plan.combine_grad(d_out, y, gate, slot_map, d_y=d_y, d_gate=d_gate)
    bad = ~torch.isfinite(d_gate)
    assert bad[0, 2].all() and bad[0, 6, 0] and bad.sum() == 3
    rows = (~torch.isfinite(d_y)).any(-1).nonzero().flatten().tolist()
    assert sorted(rows) == sorted(slot_map[0, 2].tolist() + [slot_map[0, 4, 1].item()])
    plan.close()


def test_other_stream_and_graph():
    plan, d_out, y, gate, slot_map = setup(4, 8, 30, 1032, 4)
    d_y, d_gate = torch.full_like(y, CANARY), torch.full_like(gate, CANARY)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    plan.combine_grad(d_out, y, gate, slot_map, d_y=d_y, d_gate=d_gate, stream=s)
    s.synchronize()
    check(plan, d_out, y, gate, slot_map, d_y, d_gate)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.combine_grad(d_out, y, gate, slot_map, d_y=d_y, d_gate=d_gate)
    d_out.mul_(-0.5)
    slot_map.copy_(slot_map.flatten().flip(0).view_as(slot_map))
    graph.replay()
    check(plan, d_out, y, gate, slot_map, d_y, d_gate)
    plan.close()


def test_gradient_by_differences():
    """The combine is linear in each of its inputs: its difference is the slope, up to the roundings to bf16."""
    plan, d_out, y, gate, slot_map = setup(2, 8, 12, 512, 3)
    d_y, d_gate = torch.full_like(y, CANARY), torch.full_like(gate, CANARY)
    plan.combine_grad(d_out, y, gate, slot_map, d_y=d_y, d_gate=d_gate)
    g = torch.Generator().manual_seed(4)
    v, w = torch.randn(gate.shape, generator=g).to(DEV), torch.randn(y.shape, generator=g).to(DEV)
    at = slot_map.long()

    def f(gate, y):
        return ((gate.unsqueeze(-1) * y[at]).sum(2) * d_out.double()).sum()

    gd, yd = gate.double(), y.double()
    slope = (f(gd + v.double(), yd) - f(gd - v.double(), yd)) / 2
    assert abs((d_gate.double() * v.double()).sum() - slope) <= 60 * 2.0 ** -24 * (
        (yd[at].abs() * d_out.double().abs().unsqueeze(2)).sum(-1) * v.abs()).sum()
    slope = (f(gd, yd + w.double()) - f(gd, yd - w.double())) / 2
    assert abs((d_y.double() * w.double()).sum() - slope) <= 2.0 ** -8 * (d_y.double().abs() * w.abs()).sum()
    plan.close()


def test_refusals():
    plan, d_out, y, gate, slot_map = setup(1, 2, 4, 64, 2)
    d_y, d_gate = torch.empty_like(y), torch.empty_like(gate)
    launches = plan.launches
    room = torch.empty(y.numel() + 64, device=DEV, dtype=torch.bfloat16)
    for call, message in [
        (lambda: plan.combine_grad(d_out, y, gate, slot_map), "neither"),
        (lambda: plan.combine_grad(d_out, None, gate, slot_map, d_gate=d_gate), "needs y"),
        (lambda: plan.combine_grad(d_out, y, None, slot_map, d_y=d_y), "needs gate_w"),
        (lambda: plan.combine_grad(d_out, y, gate, slot_map, d_y=d_y, d_gate=gate), "overlaps"),
        (lambda: plan.combine_grad(d_out, room[:y.numel()].view_as(y), gate, slot_map, d_y=room[64:].view_as(y)), "overlaps"),
        (lambda: plan.combine_grad(room[:256].view_as(d_out), y, gate, slot_map, d_y=room[:y.numel()].view_as(y)), "overlaps"),
        (lambda: plan.combine_grad(d_out, y, gate, slot_map, d_y=room[1:1 + y.numel()].view_as(y)), "misaligned"),
    ]:
        with pytest.raises(A.A2avError, match=message):
            call()
    assert plan.launches == launches
    plan.close()
