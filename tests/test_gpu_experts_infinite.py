"""mx_fp4_experts where single outputs leave f32's range: the other columns keep their
values, on every kernel.

One nonzero weight a row, positive tokens with large gates (SiLU(g) = g from 32 on): every
sum has one term, of few bits, so results are exact."""

import numpy as np
import pytest
import torch

import oracle
from helpers import dev, f64, mx

pytestmark = pytest.mark.gpu


# A few tokens; tiles of 128 weight rows; tiles of 256.
@pytest.mark.parametrize("T", [9, 70, 300])
@pytest.mark.parametrize("act", ["fp8", "fp4"])
def test_an_infinite_column_leaves_its_neighbours(T, act):
    print(f"experts T={T} {act}", flush=True)
    E, H, I, d = 2, 160, 96, dev()
    g = torch.Generator().manual_seed(T)
    x = torch.tensor([1.0, 1.5, 2.0, 3.0])[torch.randint(0, 4, (T, H), generator=g)].to(torch.bfloat16)
    ids = torch.randint(0, E, (T, 1), generator=g).to(torch.int32)

    up, down = torch.zeros((E, 2 * I, H)), torch.zeros((E, H, I))
    up.scatter_(2, torch.randint(0, H, (E, 2 * I, 1), generator=g), 1.0)
    up[:, :I] *= 32.0
    down.scatter_(2, torch.randint(0, I, (E, H, 1), generator=g), 1.0)
    # h >= 32: these columns overflow, upwards or downwards, the others of their 32 do not.
    down[:, 5] *= 2.0**125
    down[:, 40] *= -(2.0**125)
    down[:, 130] *= 2.0**125
    down[1, 131] *= 2.0**125
    v = [mx().mx_fp4_quantize_experts(w.to(d)) for w in (up, down)]
    y = f64(mx().mx_fp4_experts(x.to(d), ids.to(d), torch.ones((T, 1), device=d), *v, act=act))

    xh = torch.from_numpy(oracle.activation_values(f64(x), act))
    for t in range(T):
        e = int(ids[t, 0])
        a = up[e].double() @ xh[t]
        h = oracle.activation_values(oracle.bf16_round((a[:I] * a[I:]).numpy())[None], act)[0]
        o = down[e].double().numpy() @ h
        want = oracle.bf16_round(np.where(abs(o) < 2.0**128, o, np.copysign(np.inf, o)))
        assert np.isinf(want[[5, 40, 130]]).all() and np.isfinite(want[[4, 6, 41, 129]]).all()
        assert np.array_equal(y[t], want), (t, np.flatnonzero(y[t] != want))
