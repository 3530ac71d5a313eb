"""Numbers a RouteRule cannot hold are refused; nothing is cut off to fit its 32-bit fields."""
import numpy as np
import pytest

import combine_device_resident_gb300 as A


@pytest.mark.parametrize("change", [
    dict(groups=2 ** 32 + 1), dict(groups=8, groups_kept=2 ** 32 + 4), dict(groups=4, group_best=2 ** 32 + 2),
    dict(groups=2.5), dict(groups=4, groups_kept=1.5), dict(group_best=1.9), dict(groups=float("nan")),
    dict(groups=float("inf")), dict(groups="4"), dict(groups=-2 ** 31 - 1),
])
def test_numbers_that_do_not_fit_are_refused(change):
    with pytest.raises(A.A2avError, match="whole number"):
        A.RouteRule(**change)


def test_whole_numbers_of_any_type():
    r = A.RouteRule(groups=np.int64(8), groups_kept=4.0, group_best=np.float32(2.0))
    assert (r.groups, r.groups_kept, r.group_best) == (8, 4, 2)
