"""The router by scores where few candidates of a token stand close together at a border: at the last chosen expert, and at
the last kept group.  Ids are those of the 64-bit order, whatever the warp's other tokens do: a token per call."""
import numpy as np
import pytest
import torch

import combine_device_resident_gb300 as A
from tests.test_gpu_route_scores import DEV, check

pytestmark = pytest.mark.gpu


def one_token(logits, bias, k, rule):
    E = len(logits)
    plan = A.Plan(1, E, 1, 8, k, device=DEV)
    check(plan, torch.tensor(logits, dtype=torch.float32, device=DEV).view(1, 1, E), rule,
          torch.tensor(bias, dtype=torch.float32, device=DEV))
    plan.close()


def border(rng, E, ahead, pair_first):
    """Logits and biases of E experts: `ahead` clearly in front, then a single expert and two alike whose choices in 64 bits
    lie within a few steps of fp32 of each other, the two alike in front or behind, the rest far below."""
    while True:
        logits, bias = np.zeros(E, np.float32), (-1.0 - 0.01 * rng.permutation(E)).astype(np.float32)
        at = rng.permutation(E)[:ahead + 3]
        logits[at], bias[at] = 1.0, 3.0 + np.arange(ahead + 3)
        single, alike = at[0], at[1:3]
        logits[single], logits[alike] = rng.uniform(15.0, 18.0, 2)
        bias[single], bias[alike] = 0.25 + rng.integers(-8, 9, 2) * 2.0 ** -26
        s = 1.0 / (1.0 + np.exp(-logits.astype(np.float64))) + bias.astype(np.float64)
        if abs(s[single] - s[alike[0]]) > 1e-14 and (s[alike[0]] > s[single]) == pair_first:
            return logits, bias


LOW = float(torch.finfo(torch.float32).min)
WIDTHS = [(4, 0), (8, 1), (16, 0), (16, 3), (64, 7), (100, 2), (128, 0), (256, 5), (256, 0)]


def test_last_chosen_against_two_equal_ones():
    """In fp32 expert 0 leads (1.2500001 against 1.25, twice), in 64 bits expert 1 does."""
    one_token([16.86, 100.0, 100.0, 0.0], [0.25 + 3 * 2.0 ** -25, 0.25 + 2.0 ** -24, 0.25 + 2.0 ** -24, -1.0], 1,
              A.RouteRule(score="sigmoid"))


@pytest.mark.parametrize("E,ahead", WIDTHS)
def test_two_equal_ones_at_the_border(E, ahead):
    rng = np.random.default_rng(E + ahead)
    for _ in range(40):
        one_token(*border(rng, E, ahead, True), ahead + 1, A.RouteRule(score="sigmoid"))


@pytest.mark.parametrize("E,ahead", WIDTHS)
def test_one_behind_two_equal_ones_at_the_border(E, ahead):
    """fp32 may put the two alike in front, the last chosen's neighbour then says nothing about the one behind it."""
    rng = np.random.default_rng(E + ahead + 1000)
    for _ in range(40):
        one_token(*border(rng, E, ahead, False), ahead + 1, A.RouteRule(score="sigmoid"))


def test_many_equal_ones_at_the_border():
    """Five alike, of which one is chosen, and one more that belongs in front of them."""
    rng = np.random.default_rng(5)
    for E in (16, 64, 256):
        for _ in range(40):
            logits, bias = border(rng, E, 0, False)
            alike = [e for e in range(E) if (logits == logits[e]).sum() == 2]
            more = rng.permutation(np.flatnonzero(bias <= -1.0))[:3]
            logits[more], bias[more] = logits[alike[0]], bias[alike[0]]
            one_token(logits, bias, 2, A.RouteRule(score="sigmoid"))


BIG = 2.0 ** 126


@pytest.mark.parametrize("E,groups", [(16, 4), (64, 8), (256, 8), (256, 4), (24, 6), (20, 10)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("pairs", [
    [(2e38, 2e38), (3e38, 3e38)],                       # both sums past fp32's range: 64 bits tell them apart
    [(3e38, 1e38), (3e38, 2e38), (2e38, 2e38)],
    [(-3e38, -3e38), (-2e38, -2e38)],
    [(-np.inf, -np.inf), (LOW, LOW)],                   # masked by -infinity, and by the type's lowest value
    [(LOW, -np.inf), (LOW, LOW)],
    [(np.inf, -np.inf), (np.inf, 0.0), (LOW, LOW)],     # the first is no number: -infinity
    [(np.inf, 0.0), (3e38, 3e38), (np.inf, np.inf)],    # the infinite ones are equal
    [(LOW, LOW), (LOW, LOW)],
    [(BIG, BIG), (np.nextafter(np.float32(BIG), np.float32(0)), BIG)],
])
def test_sums_of_two_best_at_the_ends_of_fp32(E, groups, score, pairs):
    """Groups whose two best are these, one or two kept; the others are further down, masked, or further up."""
    size = E // groups
    rng = np.random.default_rng(E + groups)
    rest = -np.inf if min(min(p) for p in pairs) < 0 else -1.0
    for kept in (1, 2):
        for _ in range(4):
            logits = rng.standard_normal(E).astype(np.float32)
            bias = np.full((groups, size), rest, np.float32)
            for group, pair in zip(rng.permutation(groups), pairs):
                bias[group, rng.permutation(size)[:2]] = pair
            k = min(size, 3)
            one_token(logits, bias.flatten(), k, A.RouteRule(score=score, groups=groups, groups_kept=kept, group_best=2))
