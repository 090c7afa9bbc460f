"""The pairs that mx_fp4_experts takes reach its documented 2^24, short rows included."""

import pytest

from helpers import mx


@pytest.mark.parametrize("H", [32, 64, 96])
@pytest.mark.parametrize("act", [0, 1])
def test_most_pairs_of_short_rows(H, act):
    f = mx().lib().mx_fp4_experts_ws_bytes
    assert f(1 << 24, 1, 1, H, 32, act) > f((1 << 24) - 1, 1, 1, H, 32, act) - 4096 > 0
    assert f((1 << 24) + 1, 1, 1, H, 32, act) == -1
