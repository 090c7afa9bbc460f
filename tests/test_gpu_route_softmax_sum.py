"""mx_route's unnormalised softmax: weights are the float64 score's, rounded to f32 once.

Tolerance: that rounding, 2^-24 of the weight, and 2^-36 for the float64 arithmetic
before it (a term of the sum is good to 2^-42); weights under 2^-126 round to a step of
2^-149."""

import numpy as np
import pytest
import torch

import oracle
from helpers import dev, f64, mx
from test_gpu_route import logits

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("E,k", [(1, 1), (16, 16), (64, 6), (100, 64), (128, 8), (256, 8), (300, 10), (512, 64), (1024, 64)])
def test_weights_are_rounded_once(E, k, dtype):
    print(f"route E={E} k={k} {dtype}", flush=True)
    for spread in (0.01, 1.0, 20.0):
        l = (spread * logits(200, E, torch.float32, E)).to(dtype)
        l[3, E // 2 :] = float("-inf")
        ids, w = mx().mx_route(l.to(dev()), k, renorm=False, scale=3.0)
        rid, rw = oracle.route_ref(f64(l), k, renorm=False, scale=3.0)
        assert np.array_equal(ids.cpu().numpy(), rid), "ids"
        err = np.abs(f64(w) - rw)
        assert (err <= rw * (2.0**-24 + 2.0**-36) + 2.0**-150).all(), np.nanmax(err / rw) * 2.0**24


@pytest.mark.parametrize("E,k", [(64, 64), (256, 8), (600, 64)])
def test_a_bias_of_zeros_leaves_the_weights(E, k):
    l = logits(300, E, torch.float32, E).to(dev())
    ids, w = mx().mx_route(l, k, renorm=False)
    ib, wb = mx().mx_route(l, k, bias=torch.zeros(E, device=dev()), renorm=False)
    same = ids == ib  # (scores that are equal in f32 change places)
    assert same.float().mean() > 0.99 and torch.equal(w[same], wb[same])
