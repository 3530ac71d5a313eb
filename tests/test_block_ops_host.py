"""The router by scores, the gradients and the norms around a block, what needs no GPU: refusals of the
C ABI and of the binding; nothing is enqueued."""
import ctypes

import pytest
import torch

import combine_device_resident_gb300 as A
from combine_device_resident_gb300 import binding


@pytest.fixture(scope="module")
def lib():
    from combine_device_resident_gb300 import build

    build.build()
    return A.load_library()


def _plan(**kw):
    """A Plan's Python side without a device: argument checks run before the handle is used."""
    p = object.__new__(A.Plan)
    p.lib = A.load_library()
    p.device = torch.device("cpu")
    p.R, p.E, p.T, p.H, p.k = 2, 4, 3, 32, 2
    p.arena_rows = 12
    p.handle = None
    p._s = lambda stream: None
    p.__dict__.update(kw)
    return p


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def _f(*shape):
    return torch.zeros(shape)


def _i(*shape):
    return torch.zeros(shape, dtype=torch.int32)


def test_null_plan_is_refused(lib):
    rule = A.RouteRule()
    norm = binding.BlockNormArgs()
    assert lib.a2av_route_scores(None, rule, 16, None, 32, 48, None) == 1
    assert lib.a2av_route_scores_grad(None, rule, 16, 32, 48, 64, None) == 1
    assert lib.a2av_combine_grad(None, 16, 16, 16, 16, None, 16, None) == 1
    assert b"pointer" in lib.a2av_last_error()
    assert lib.a2av_block_norm(None, norm, 16, 16, 16, None, None, None) == 1
    assert lib.a2av_block_norm_grad(None, norm, 16, 16, None, 16, 16, 16, None, None, None, None, None) == 1
    assert b"pointer" in lib.a2av_last_error()
    assert lib.a2av_norm_scratch_bytes(None) == -1


@pytest.mark.parametrize("change,message", [
    (dict(gate_kind=4), b"gate_kind"), (dict(gate_kind=-1), b"gate_kind"), (dict(gate_kind=1), b"go together"),
    (dict(gate=16), b"go together"), (dict(gate=8, gate_kind=1), b"misaligned"), (dict(post_weight=2), b"misaligned"),
    (dict(eps=-1.0), b"eps"), (dict(eps=float("nan")), b"eps"), (dict(residual_scale=float("inf")), b"scales"),
    (dict(branch_scale=float("nan")), b"scales"),
])
def test_weights_of_the_block_norm_are_refused(lib, change, message):
    n = binding.BlockNormArgs(None, None, None, 0, 1.0, 1.0, 1e-6)
    for name, v in change.items():
        setattr(n, name, v)
    assert lib.a2av_block_norm(None, n, 16, 16, 16, None, None, None) == 1
    assert message in lib.a2av_last_error()
    assert lib.a2av_block_norm_grad(None, n, 16, 16, None, 16, 16, 16, None, None, None, None, None) == 1
    assert message in lib.a2av_last_error()
    assert lib.a2av_block_norm(None, None, 16, 16, 16, None, None, None) == 1


def test_rule():
    r = A.RouteRule(score="sigmoid", groups=8, groups_kept=4, group_best=2, renormalize=False, scale=2.5)
    assert (r.score, r.groups, r.groups_kept, r.group_best, r.renormalize, r.scale) == (1, 8, 4, 2, 0, 2.5)
    assert A.RouteRule(groups=4).groups_kept == 4
    with pytest.raises(A.A2avError, match="score"):
        A.RouteRule(score="relu")
    # the header's struct, in its order
    assert [f[0] for f in A.RouteRule._fields_] == ["score", "groups", "groups_kept", "group_best", "renormalize", "scale"]
    assert ctypes.sizeof(A.RouteRule) == 24
    assert ctypes.sizeof(binding.BlockNormArgs) == 40


def test_binding_checks_shapes_and_types(lib):
    p, rule = _plan(), A.RouteRule()
    x, row, half = _bf(2, 3, 32), _bf(32), _f(32)
    cases = [
        (lambda: p.route_scores(_f(2, 3, 5), _i(2, 3, 2), _f(2, 3, 2), rule), "logits has shape"),
        (lambda: p.route_scores(_bf(2, 3, 4), _i(2, 3, 2), _f(2, 3, 2), rule), "logits must be"),
        (lambda: p.route_scores(_f(2, 3, 4), _f(2, 3, 2), _f(2, 3, 2), rule), "topk_idx must be"),
        (lambda: p.route_scores(_f(2, 3, 4), _i(2, 3, 2), _f(2, 3, 1), rule), "gate_w has shape"),
        (lambda: p.route_scores(_f(2, 3, 4), _i(2, 3, 2), _f(2, 3, 2), rule, bias=_f(5)), "bias has shape"),
        (lambda: p.route_scores(_f(2, 3, 4), _i(2, 3, 2), _f(2, 3, 2), "sigmoid"), "RouteRule"),
        (lambda: p.route_scores(_f(2, 3, 8)[..., ::2], _i(2, 3, 2), _f(2, 3, 2), rule), "contiguous"),
        (lambda: p.route_scores_grad(_f(2, 3, 4), _i(2, 3, 2), _f(2, 3, 2), _f(2, 3, 2), rule), "d_logits has shape"),
        (lambda: p.route_scores_grad(_f(2, 3, 4), _i(2, 3, 2), _f(2, 3), _f(2, 3, 4), rule), "d_gate has shape"),
        (lambda: p.combine_grad(_bf(2, 3, 31), _bf(12, 32), _f(2, 3, 2), _i(2, 3, 2), d_y=_bf(12, 32)), "d_out has"),
        (lambda: p.combine_grad(x, _bf(11, 32), _f(2, 3, 2), _i(2, 3, 2), d_y=_bf(12, 32)), "y has shape"),
        (lambda: p.combine_grad(x, _bf(12, 32), _f(2, 3, 2), _i(2, 3, 2), d_gate=_bf(2, 3, 2)), "d_gate must be"),
        (lambda: p.combine_grad(x, _bf(12, 32), _f(2, 3, 2), _f(2, 3, 2), d_gate=_f(2, 3, 2)), "slot_map must be"),
        (lambda: p.block_norm(x, _bf(2, 3, 31), residual_out=x), "residual has shape"),
        (lambda: p.block_norm(x, x, residual_out=x, post_weight=half), "post_weight must be"),
        (lambda: p.block_norm(x, x, residual_out=x, gate=_bf(3, 32)), "gate has shape"),
        (lambda: p.block_norm(x, x, residual_out=x, gate=torch.tensor(1.0)), "gate must be a tensor"),
        (lambda: p.block_norm(x, x, residual_out=x, gate=2.0), "gate must be a tensor"),
        (lambda: p.block_norm(x, x, y=_bf(2, 3, 16), weight=row), "y has shape"),
        (lambda: p.block_norm(x, x, rows8=torch.zeros(2, 3, 32, dtype=torch.uint8), weight=row), "rows8 has shape"),
        (lambda: p.block_norm_grad(x, x, x, _bf(2, 3), d_y=x, weight=row), "d_residual has shape"),
        (lambda: p.block_norm_grad(x, x, x, x, d_y=x, weight=row, d_weight=row), "d_weight must be"),
        (lambda: p.block_norm_grad(x, x, x, x, d_y=x, weight=row, d_gate=half), "d_gate needs gate"),
        (lambda: p.block_norm_grad(x, x, x, x, d_y=x, gate=_bf(2, 32), d_gate=half), "d_gate has shape"),
        (lambda: p.block_norm_grad(x, x, x, x, d_y=x, gate=x, d_gate=_f(2, 3, 32)), "d_gate must be"),
    ]
    for call, message in cases:
        with pytest.raises(A.A2avError, match=message):
            call()
