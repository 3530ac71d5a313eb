"""The norm and the experts' products, what needs no GPU: refusals of the C
ABI and of the binding (nothing is enqueued), and the weight layouts."""
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


def test_null_plan_is_refused(lib):
    assert lib.a2av_rms_norm(None, 16, None, 16, 1e-6, None, 16, None, None) == 1
    assert lib.a2av_quantize_rows(None, 16, 16, None, 16, None) == 1
    assert lib.a2av_expert_matmul(None, 16, 16, None, 16, 8, 8, 0, 0, 0, None, None) == 1
    assert b"pointer" in lib.a2av_last_error()


def test_unknown_weight_type_and_activation_are_refused(lib):
    assert lib.a2av_expert_matmul(None, 16, 16, None, 16, 8, 8, 3, 0, 0, None, None) == 1
    assert b"weight_type" in lib.a2av_last_error()
    assert lib.a2av_expert_matmul(None, 16, 16, None, 16, 8, 8, 0, 0, 2, None, None) == 1
    assert b"activation" in lib.a2av_last_error()


def _plan(**kw):
    """A Plan's Python side without a device: argument checks run before the handle is used."""
    p = object.__new__(A.Plan)
    p.lib = A.load_library()
    p.device = torch.device("cpu")
    p.R, p.E, p.T, p.H, p.k = 2, 4, 3, 32, 1
    p.arena_rows = 6
    p.handle = None
    p.recv_order = "expert"
    p.__dict__.update(kw)
    return p


def _bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_binding_checks_shapes_and_types(lib):
    p = _plan()
    sp = A.Splits(2, 4, "cpu")
    x, w, y = _bf(6, 32), _bf(4, 16, 32), _bf(6, 16)
    cases = [
        (lambda: p.rms_norm(_bf(2, 3, 31), _bf(32), y=_bf(2, 3, 32)), "x has shape"),
        (lambda: p.rms_norm(_bf(2, 3, 32), _bf(31), y=_bf(2, 3, 32)), "weight has shape"),
        (lambda: p.rms_norm(_bf(2, 3, 32), _bf(32), rows8=_bf(2, 3, 48)), "rows8 must be"),
        (lambda: p.rms_norm(_bf(2, 3, 32), _bf(32), rows8=torch.zeros(2, 3, 32, dtype=torch.uint8)), "rows8 has shape"),
        (lambda: p.rms_norm(_bf(2, 3, 32).float(), _bf(32), y=_bf(2, 3, 32)), "x must be"),
        (lambda: p.rms_norm(_bf(2, 3, 64)[..., ::2], _bf(32), y=_bf(2, 3, 32)), "contiguous"),
        (lambda: p.quantize_rows(_bf(5, 32), sp, torch.zeros(6, 48, dtype=torch.uint8)), "x has shape"),
        (lambda: p.quantize_rows(x, sp, torch.zeros(6, 47, dtype=torch.uint8)), "rows8 has shape"),
        (lambda: p.quantize_rows(x, A.Splits(2, 8, "cpu"), torch.zeros(6, 48, dtype=torch.uint8)), "splits were made"),
        (lambda: p.expert_matmul(x, _bf(3, 16, 32), sp, y), "w has shape"),
        (lambda: p.expert_matmul(x, w, sp, _bf(6, 8)), "w has shape"),
        (lambda: p.expert_matmul(x, w, sp, y, activation="swiglu"), "w has shape"),
        (lambda: p.expert_matmul(x, w, sp, y, activation="gelu"), "activation"),
        (lambda: p.expert_matmul(_bf(6, 24), w, sp, y), "x has shape"),
        (lambda: p.expert_matmul(x, w.float(), sp, y), "w must be"),
        (lambda: p.expert_matmul(x, w, None, y), "Splits"),
        (lambda: p.expert_matmul(x, w.to(torch.float8_e4m3fn), sp, y), "x must be"),
        (lambda: p.expert_matmul_w4(x, torch.zeros(4, 16, 4, dtype=torch.int32), _bf(4, 16, 3), sp, y), "groups"),
        (lambda: p.expert_matmul_w4(x, torch.zeros(4, 16, 4, dtype=torch.int32), _bf(4, 8, 1), sp, y), "w_scale has"),
        (lambda: p.expert_matmul_w4(x, torch.zeros(4, 16, 4), _bf(4, 16, 1), sp, y), "w must be"),
    ]
    for call, message in cases:
        with pytest.raises(A.A2avError, match=message):
            call()


def test_quantized_weights_are_within_half_a_step():
    g = torch.Generator().manual_seed(1)
    w = torch.randn(3, 5, 64, generator=g)
    w[1, 2] = 0.0
    q, s = A.quantize_weights(w)
    # e4m3: half a step is 2^-4 of the value, 2^-10 of the scale below the smallest normal 2^-6
    assert ((q.float() * s[..., None] - w).abs() <= w.abs() * 2 ** -4 + s[..., None] * 2 ** -10 + 1e-12).all()
    assert (q[1, 2].float() == 0).all() and s[1, 2] == 0


@pytest.mark.parametrize("group", [32, 64, 128])
def test_w4_words_come_back(group):
    g = torch.Generator().manual_seed(2)
    w = torch.randn(2, 6, 256, generator=g)
    w[0, 1, :group] = 0.0
    words, s = A.pack_weights_w4(w, group)
    assert words.shape == (2, 6, 32) and words.dtype == torch.int32 and s.shape == (2, 6, 256 // group)
    v = A.unpack_weights_w4(words, s)
    # a step is the scale, max|w| / 7 rounded to bf16: half a step, and the maximum may be cut by the scale's rounding
    s32 = s.float().repeat_interleave(group, -1)
    assert ((v - w).abs() <= s32 * (0.5 + 8 * 2 ** -8)).all()
    # the layout itself: bit 4*(k//2) + 16*(k%2) of word k//8
    k = 37
    q = (int(words[1, 3, k // 8]) >> (4 * ((k % 8) // 2) + 16 * (k % 2))) & 15
    assert (q - 8) * float(s[1, 3, k // group]) == float(v[1, 3, k])


def test_pack_weights_w4_refuses_other_groups():
    for group, K in ((48, 96), (128, 64), (16, 64)):
        with pytest.raises(A.A2avError, match="group"):
            A.pack_weights_w4(torch.zeros(2, K), group)


def test_rows8_parts_are_views():
    rows8 = torch.zeros(2, 3, 48, dtype=torch.uint8)
    q, s = A.rows8_parts(rows8)
    assert q.shape == (2, 3, 32) and s.shape == (2, 3)
    s[1, 2] = 2.0
    assert rows8[1, 2, 32:36].view(torch.float32).item() == 2.0


def test_new_calls_have_signatures(lib):
    for name in ("a2av_rms_norm", "a2av_quantize_rows", "a2av_expert_matmul"):
        assert getattr(lib, name).restype is ctypes.c_int32
        assert name in binding.EXPORTED
