"""mx_block_norm_slab's residual_scale is a float64 like the formula's: scales that f32
cannot hold, in every form of the kernel.

Tolerance: h's float64 product and sum are off by 2^-52 of their terms' magnitudes here
and in the kernel, so h lies between the roundings (f32, then the residual's type) of the
ends of a range of 2^-50 of them: either neighbour of a tie that the two sides cannot tell
from it, as 0.1 r + x makes many of (0.1 is 1 / 10 to 2^-54 of itself, so with r a multiple
of 5 the sum is a tie to within that), and else one value. A scale rounded to f32 would
move h by up to 2^-24 of the residual's term before its rounding."""

import math

import numpy as np
import pytest
import torch

from helpers import dev, f64, mx
from test_gpu_block_norm import BF16, F32, between

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("alpha", [0.1, 1.0 / 3.0, 0.22, -0.7, 1.4 / math.sqrt(40.0), 1e-30])
@pytest.mark.parametrize("rdt", [BF16, F32])
@pytest.mark.parametrize("M,K", [(3, 192), (40, 5120), (2, 32768), (2049, 1088)])
def test_scales_that_f32_cannot_hold(M, K, rdt, alpha):
    print(f"block norm {M}x{K} {rdt} residual_scale {alpha}", flush=True)
    d = dev()
    g = torch.Generator(device=d).manual_seed(M + K)
    x = torch.randn((M, K), generator=g, device=d).to(BF16)
    r = (3.0 * torch.randn((M, K), generator=g, device=d)).to(rdt)
    _, h = mx().mx_block_norm_slab(x, r, residual_scale=alpha)
    a, n = alpha * f64(r), f64(x)
    between(f64(h), a + n, (np.abs(a) + np.abs(n)) * 2.0**-50, rdt, "h")
