"""The norms' gradient where ranks have no tokens: their gate rows, and whatever else belongs to them alone, may hold
anything."""
import pytest
import torch

import combine_device_resident_gb300 as A
from tests.test_gpu_block_norm import DEV, check_grad, inputs, run_grad

pytestmark = pytest.mark.gpu
ODD = [float("nan"), float("inf")]


@pytest.mark.parametrize("odd", ODD)
@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("R,T,H", [(4, 6, 48), (4, 6, 1040), (40, 3, 264), (4, 3, 8200), (64, 40, 512)])
def test_gates_of_ranks_without_tokens(R, T, H, post, odd):
    plan = A.Plan(R, R, T, H, 1, device=DEV)
    n = torch.arange(R, dtype=torch.int32, device=DEV) % 3 - 1  # none, none, one
    n[-1] = T + 3
    plan.set_active_tokens(n)
    live = torch.arange(T, device=DEV).view(1, T) < n.view(R, 1)
    i = inputs(R, T, H, post, "rank", 5)
    dead = n <= 0
    for name in ("x", "residual", "d_y", "d_residual_out"):
        i[name][~live] = odd
    filled = dict(i, gate=i["gate"].clone())
    filled["gate"][dead] = odd
    scratch = plan.new_norm_scratch()
    got, want = run(plan, filled, scratch), run_grad(plan, i, "rank", live=live, scratch=scratch)
    check_grad(i, got, 1.0, 1.0, ("d_y", "d_residual_out"), live)
    assert all(torch.equal(got[k], want[k]) for k in got if got[k] is not None)
    assert (got["d_gate"][dead] == 0).all()
    plan.close()


def run(plan, i, scratch):
    """The call alone."""
    H = plan.H
    out = dict(d_x=torch.full_like(i["x"], 7.0), d_residual=torch.full_like(i["x"], 7.0),
               d_weight=torch.full((H,), 7.0, device=DEV),
               d_post=torch.full((H,), 7.0, device=DEV) if i["post_weight"] is not None else None,
               d_gate=None if i["gate"] is None else torch.full(i["gate"].shape, 7.0, device=DEV))
    plan.block_norm_grad(i["x"], i["residual"], out["d_x"], out["d_residual"], weight=i["weight"], d_y=i["d_y"],
                         d_residual_out=i["d_residual_out"], post_weight=i["post_weight"], gate=i["gate"],
                         d_weight=out["d_weight"], d_post_weight=out["d_post"], d_gate=out["d_gate"], scratch=scratch)
    return out


@pytest.mark.parametrize("odd", ODD)
@pytest.mark.parametrize("gate", ["channel", "rank"])
@pytest.mark.parametrize("H", [48, 8200])
def test_weights_without_any_token(gate, H, odd):
    """A sum over no tokens is zero, whatever the weights hold."""
    plan = A.Plan(2, 2, 5, H, 1, device=DEV)
    plan.set_active_tokens(torch.zeros(2, dtype=torch.int32, device=DEV))
    i = {name: torch.full_like(t, odd) for name, t in inputs(2, 5, H, True, gate).items()}
    got = run(plan, i, plan.new_norm_scratch())
    assert all((got[name] == 0).all() for name in ("d_weight", "d_post", "d_gate"))
    plan.close()
