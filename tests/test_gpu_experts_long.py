"""mx_fp4_experts on the longest rows, where a step left out or read from a wrong place has
to show: one nonzero weight a row, in the first, a middle or one of the last steps, and
positive tokens with large gates (SiLU(g) = g from 32 on). Every sum then has one term, of
few bits, so all results are exact; and each row of the down product is one product of its
own, so a lost step is a row of zeros. Beyond 4 GiB of weights: bit for bit the result of
the same slabs alone, in tiles of 256 weight rows."""

import numpy as np
import pytest
import torch

import oracle
import synth
from helpers import dev, f64, mx

pytestmark = pytest.mark.gpu


def columns(K, E, N, g):
    """A column for each row: the ends of the first and the last four steps of 128, the
    middle, then any."""
    named = [c for s in (0, 1, K // 256, K // 128 - 4, K // 128 - 3, K // 128 - 2, K // 128 - 1) if s >= 0
             for c in (128 * s, 128 * s + 31, 128 * s + 64, 128 * s + 127) if 0 <= c < K] + [0, K - 1]
    c = torch.randint(0, K, (E, N), generator=g)
    for e in range(E):
        order = torch.randperm(N, generator=g)[: len(named)]
        c[e, order] = torch.tensor(named)[torch.randperm(len(named), generator=g)][: len(order)]
    return c[..., None]


def sparse(E, N, K, g):
    w = torch.zeros((E, N, K))
    return w.scatter_(2, columns(K, E, N, g), torch.where(torch.rand((E, N, 1), generator=g) < 0.5, 1.0, 2.0))


# A few tokens; tiles of 128 weight rows; of 256.
@pytest.mark.parametrize("T", [3, 16, 70, 200])
@pytest.mark.parametrize("act", ["fp8", "fp4"])
@pytest.mark.parametrize("H,I", [(65536, 32), (32, 65536), (16416, 160), (160, 16416)])
def test_no_step_is_lost(H, I, T, act):
    print(f"experts T={T} H={H} I={I} {act}", flush=True)
    E, d = 2, dev()
    g = torch.Generator().manual_seed(T + H)
    x = torch.tensor([1.0, 1.5, 2.0, 3.0])[torch.randint(0, 4, (T, H), generator=g)].to(torch.bfloat16)
    ids = (torch.arange(T) % E).to(torch.int32)[:, None]
    up, down = sparse(E, 2 * I, H, g), sparse(E, H, I, g)
    up[:, :I] *= 32.0
    v = [mx().mx_fp4_quantize_experts(w.to(d)) for w in (up, down)]
    y = f64(mx().mx_fp4_experts(x.to(d), ids.to(d), torch.ones((T, 1), device=d), *v, act=act))

    xh = oracle.activation_values(f64(x), act)

    def rows(w, v):  # v @ w.T, one term a row
        c = w.argmax(dim=1).numpy()
        return v[:, c] * w.numpy()[np.arange(len(c)), c]

    for e in range(E):
        t = np.flatnonzero(ids[:, 0].numpy() == e)
        a = rows(up[e], xh[t])
        h = oracle.activation_values(oracle.bf16_round(a[:, :I] * a[:, I:]), act)
        want = oracle.bf16_round(rows(down[e], h))
        bad = y[t] != want
        assert not bad.any(), (e, int(bad.sum()), np.unique(np.flatnonzero(bad.any(0)))[:8])


def test_large_tiles_past_4_gib():
    # Codes of 4.7 and 2.3 GiB; a first and the last expert take the pairs in turn (64 and
    # more for each of the 300 on average), and the same two alone as two experts.
    E, H, I, T, d = 300, 4096, 4096, 19213, dev()
    g = torch.Generator(device=d).manual_seed(2)

    def big(N, K):
        sq, ss = ((K + 127) // 128, N // 16, 4, 16, 16), ((K + 127) // 128, N, 4)
        q = torch.empty((E,) + sq, dtype=torch.uint8, device=d)
        for e in range(E):
            q[e] = torch.randint(0, 256, sq, generator=g, device=d, dtype=torch.uint8)
        return mx().FP4Experts(q, torch.full((E,) + ss, 120, dtype=torch.uint8, device=d), N, K)

    up, down = big(2 * I, H), big(H, I)
    assert up.q.numel() > 1 << 32 and T >= 64 * E
    pick = torch.tensor([0, E - 1], device=d)
    two = [mx().FP4Experts(t.q[pick].contiguous(), t.s[pick].contiguous(), t.rows, t.K) for t in (up, down)]
    x = synth.make_activation(T, H, seed=1).to(d)
    ids = (torch.arange(T, device=d, dtype=torch.int32) % 2)[:, None]
    w = torch.ones((T, 1), device=d)
    for act in ("fp8", "fp4"):
        y = mx().mx_fp4_experts(x, ids * (E - 1), w, up, down, act=act)
        assert torch.equal(y, mx().mx_fp4_experts(x, ids, w, *two, act=act)), act
