"""The block norm's reference keeps a residual scale that f32 cannot hold."""

import numpy as np
import pytest

import oracle


@pytest.mark.parametrize("alpha", [0.1, 1.0 / 3.0, 0.75])
def test_scale_is_not_rounded(alpha):
    h, mag = oracle.block_h_ref(np.zeros((1, 2)), np.array([[1.0, -2.0]]), residual_scale=alpha)
    assert h.tolist() == [[alpha, -2.0 * alpha]] and mag.tolist() == [[alpha, 2.0 * alpha]]
