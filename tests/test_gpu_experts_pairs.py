"""mx_fp4_experts with the most pairs that it takes, and with tokens' codes past 2 GiB
(13.4 million rows of 160 columns: 3.4e9 bytes): rows are those of a smaller call on the same
kernel."""

import pytest
import torch

from helpers import dev, mx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,H", [(1 << 24, 32), ((1 << 31) // 160, 160)])
@pytest.mark.parametrize("act", ["fp8", "fp4"])
def test_most_pairs(T, H, act):
    E, I, d = 3, 32, dev()
    print(f"experts T={T} H={H} {act}", flush=True)
    g = torch.Generator(device=d).manual_seed(1)
    x = torch.randn((T, H), generator=g, device=d).to(torch.bfloat16)
    ids = torch.randint(0, E, (T, 1), generator=g, device=d, dtype=torch.int32)
    w = torch.rand((T, 1), generator=g, device=d)
    up, down = (mx().mx_fp4_quantize_experts(0.3 * torch.randn(s, generator=g, device=d)) for s in ((E, 2 * I, H), (E, H, I)))
    y = mx().mx_fp4_experts(x, ids, w, up, down, act=act)
    n = 5000
    for t in (0, T // 2 - 17, T - n):
        s = slice(t, t + n)
        assert torch.equal(y[s], mx().mx_fp4_experts(x[s], ids[s], w[s], up, down, act=act)), t
