"""A mixture-of-experts feed-forward block as a program runs it: block norm, router
logits, mx_route, mx_fp4_experts, and the block norm whose slab the next linear reads;
eagerly, and replayed from a graph with other inputs."""

import numpy as np
import pytest
import torch

import oracle
import synth
from helpers import dev, f64, mx
from test_gpu_experts import values, weights

pytestmark = pytest.mark.gpu

E, K, H, I, N = 12, 3, 256, 160, 192


class Block:
    def __init__(self):
        g = torch.Generator().manual_seed(1)
        d = dev()
        rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
        self.router = (rn(E, H) / 16).to(d)
        self.bias = (0.1 * rn(E)).to(d)
        self.gain, self.post, self.next = ((1 + 0.1 * rn(H)).to(d) for _ in range(3))
        self.gate = torch.full((H,), 0.5, device=d)
        (self.up, self.uw), (self.down, self.dw) = weights(E, 2 * I, H, 2), weights(E, H, I, 3)
        self.w = mx().mx_fp4_quantize_weight_slab(synth.make_weight(N, H, seed=4).to(d))

    def __call__(self, attn, residual):
        y, h = mx().mx_block_norm_slab(attn, residual, weight=self.gain, act=None)
        logits = torch.mm(y.float(), self.router.t())
        ids, w = mx().mx_route(logits, K, scores="sigmoid", bias=self.bias, groups=4, top_groups=2, scale=1.5)
        o = mx().mx_fp4_experts(y, ids, w, self.up, self.down)
        slab, h2 = mx().mx_block_norm_slab(o, h, post=True, post_weight=self.post, gate=self.gate, weight=self.next)
        return {"y": y, "h": h, "logits": logits, "ids": ids, "w": w, "o": o, "h2": h2,
                "out": mx().mx_fp4_linear_slab(slab, self.w)}


@pytest.mark.parametrize("T", [1, 12, 75, 700])
def test_block_stage_by_stage_and_replayed(T):
    print(f"moe block T={T}", flush=True)
    d = dev()
    b = Block()
    ins = [(synth.make_activation(T, H, seed=s).to(d), (3.0 * torch.randn((T, H), generator=torch.Generator().manual_seed(s))).to(d))
           for s in (5, 6, 7)]
    r = b(*ins[0])
    ids, w = oracle.route_ref(f64(r["logits"]), K, scores="sigmoid", bias=f64(b.bias), groups=4, top_groups=2, scale=1.5)
    assert np.array_equal(r["ids"].cpu().numpy(), ids)
    assert (np.abs(f64(r["w"]) - w) <= 2.0**-23 * np.abs(w)).all()
    ref, tol = oracle.experts_ref(f64(r["y"]), ids, f64(r["w"]), values(b.uw), values(b.dw), "fp8", "silu")
    assert (np.abs(f64(r["o"]) - ref) <= tol).all()
    hv, mag = oracle.block_h_ref(f64(r["o"]), f64(r["h"]), 1.0, True, f64(b.post), f64(b.gate))
    assert (np.abs(f64(r["h2"]) - hv) <= 2.0**-20 * mag).all()

    a, res = ins[0][0].clone(), ins[0][1].clone()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = b(a, res)
    for x, h in ins + ins[:1]:
        want = b(x, h)
        a.copy_(x)
        res.copy_(h)
        g.replay()
        torch.cuda.synchronize()
        for name in ("ids", "w", "o", "h2", "out"):
            assert torch.equal(got[name], want[name]), name
    del g
