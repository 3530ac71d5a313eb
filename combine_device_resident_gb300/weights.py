"""Laying out expert weights once, before serving, and looking into 8-bit rows.

Plain torch on whatever device the tensors are on; nothing here runs per step.
"""
from __future__ import annotations

from .binding import ROW8_TAIL, A2avError

# Bit of weight k % 8 in its word: even k in the low half, odd k in the high half, so that one mask
# takes two neighbours out as the two halves of a register.
W4_SHIFTS = (0, 16, 4, 20, 8, 24, 12, 28)
E4M3_MAX = 448.0
ZERO_ROW = 1e-30  # as in the 8-bit rows the kernels write


def quantize_weights(w):
    """(float8_e4m3fn [..][K], fp32 scale [..]) of w [..][K]: scale = max|w| / 448 per row; a row whose
    maximum is below 1e-30 is zeros with scale 0 (448 / max|w| has to lie in fp32's range)."""
    import torch

    w = w.float()
    a = w.abs().amax(-1)
    zero = a < ZERO_ROW  # false for NaN
    inv = torch.where(zero, 0.0, E4M3_MAX / a)
    q = (w * inv.unsqueeze(-1)).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)
    return q, torch.where(zero, 0.0, a / E4M3_MAX)


def pack_weights_w4(w, group: int = 128):
    """(int32 words [..][K/8], bf16 scales [..][K/group]) of w [..][K].

    A weight is (q - 8) * scale with q in 0..15; the scale is max|w| / 7 of its
    group, rounded to bf16 before the weights are divided by it."""
    import torch

    K = w.shape[-1]
    if group not in (32, 64, 128) or K % group:
        raise A2avError(f"group must be 32, 64 or 128 and divide K, got {group} and K = {K}")
    v = w.float().unflatten(-1, (K // group, group))
    scale = (v.abs().amax(-1) / 7.0).to(torch.bfloat16)
    s = scale.float().unsqueeze(-1)
    q = torch.where(s > 0, v / s, torch.zeros_like(v)).round_().clamp_(-8, 7).to(torch.int64) + 8
    q = q.flatten(-2).unflatten(-1, (K // 8, 8))
    words = (q << torch.tensor(W4_SHIFTS, dtype=torch.int64, device=w.device)).sum(-1)
    return torch.where(words >= 2 ** 31, words - 2 ** 32, words).to(torch.int32), scale


def unpack_weights_w4(words, scale):
    """fp32 weights [..][K] that (words, scale) stand for."""
    import torch

    q = (words.unsqueeze(-1) >> torch.tensor(W4_SHIFTS, dtype=torch.int32, device=words.device)) & 15
    v = (q - 8).flatten(-2).float()
    return v * scale.float().repeat_interleave(v.shape[-1] // scale.shape[-1], dim=-1)


def rows8_parts(rows8):
    """Views of 8-bit rows [..][K+16]: (float8_e4m3fn values [..][K], fp32 scales [..])."""
    import torch

    K = rows8.shape[-1] - ROW8_TAIL
    return rows8[..., :K].view(torch.float8_e4m3fn), rows8[..., K:K + 4].view(torch.float32)[..., 0]
