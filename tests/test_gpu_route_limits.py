"""mx_route at the most tokens that it takes, with a team of 64 lanes a token."""

import pytest
import torch

from helpers import dev, mx

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1 << 26, (1 << 26) - 3])
def test_most_tokens_of_many_experts(T):
    E, d = 257, dev()
    print(f"route T={T} E={E}", flush=True)
    want = torch.arange(T, device=d, dtype=torch.int32) % E
    logits = torch.zeros((T, E), dtype=torch.bfloat16, device=d)  # 34.5 GB
    logits.scatter_(1, want.long()[:, None], 1.0)
    ids, w = mx().mx_route(logits, 1)
    assert torch.equal(ids[:, 0], want) and (w == 1.0).all()
