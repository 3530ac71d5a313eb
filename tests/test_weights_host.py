"""Weight layouts at the ends of their range (no GPU)."""
import torch

import combine_device_resident_gb300 as A


def test_rows_of_the_smallest_weights_become_zeros_not_nan():
    """448 / max|w| is past fp32 for a maximum below 1.3e-36: such a row, as an 8-bit row of the norm (below 1e-30), is
    zeros with scale 0."""
    w = torch.zeros(4, 32)
    w[0, 3], w[0, 4] = 1e-37, -3e-38
    w[1, 5] = 1e-45
    w[2, 6] = 9e-31
    w[3, 7], w[3, 8] = 2e-30, -1e-30
    q, s = A.quantize_weights(w)
    assert (q[:3].float() == 0).all() and (s[:3] == 0).all()
    back = q.float() * s[:, None]
    # half a step of e4m3, and of the fp32 factors
    assert ((back - w)[3].abs() <= w[3].abs() * (2 ** -4 + 2 ** -22)).all() and (q[3, :7].float() == 0).all()


def test_nan_and_infinite_weights_stay_in_their_row():
    w = torch.ones(3, 32)
    w[0, 1], w[1, 1] = float("nan"), float("inf")
    q, s = A.quantize_weights(w)
    assert torch.isnan(s[0]) and torch.isinf(s[1]) and torch.isnan(q[1, 1].float())
    assert (q[2].float() * s[2] == 1).all()
    words, scale = A.pack_weights_w4(w, 32)
    back = A.unpack_weights_w4(words, scale)
    assert torch.isnan(back[0]).all() and not torch.isfinite(back[1]).any() and (back[2] - 1).abs().max() < 0.01
