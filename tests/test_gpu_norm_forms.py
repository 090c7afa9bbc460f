"""mx_rmsnorm_slab in both its forms (one row a block; tiles of eight rows, from
2048 rows at K <= 2048 and 32768 rows past it) on special values in every operand,
in captured graphs and on two streams. Comparisons are bit for bit, as in
test_gpu_norm.py."""

import pytest
import torch

import synth
from helpers import dev, mx
from test_gpu_norm import bits, check

pytestmark = pytest.mark.gpu


def special(K, rdtype):
    """Rows of x and of the residual that overflow, cancel, vanish or are not finite."""
    big = torch.finfo(torch.bfloat16).max
    x = synth.make_activation(14, K, seed=K)
    r = torch.randn((14, K), generator=torch.Generator().manual_seed(K)).to(rdtype)
    r[0] = -x[0].to(rdtype)  # h = 0
    x[1], r[1] = big, big  # h overflows
    x[2], r[2] = big, -big
    x[3, 1], r[3, 1] = float("inf"), float("-inf")
    r[4, K - 1] = float("nan")
    r[5, 0] = float("inf")
    x[6], r[6] = 2.0**-133, torch.finfo(rdtype).tiny  # subnormal and the smallest normal
    x[7], r[7] = -0.0, -0.0
    x[8], r[8] = 0.0, torch.finfo(rdtype).smallest_normal * torch.finfo(rdtype).eps  # the smallest subnormal
    r[9] = 256 * x[9].to(rdtype) + 1  # sums that round in bf16
    x[10], r[10] = big, torch.finfo(rdtype).max
    x[11, ::3] = -big
    r[12] *= 1e30
    r[13] *= 1e-30
    return x, r


@pytest.mark.parametrize("act", ["fp8", "fp4"])
@pytest.mark.parametrize("rdtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M", [14, 2062])
def test_special_rows_of_residual_and_gain(M, rdtype, act):
    print(f"norm special M={M} {rdtype} {act}", flush=True)
    d = dev()
    K = 192
    x, r = special(K, rdtype)
    x, r = x.repeat((M + 13) // 14, 1)[:M], r.repeat((M + 13) // 14, 1)[:M]
    for wdtype, values in ((torch.float32, (0.0, -0.0, 1e38, 1e-45, -3.0)), (torch.bfloat16, (float("nan"),)),
                           (torch.float32, (float("inf"),))):
        w = 1 + 0.2 * torch.randn((K,), generator=torch.Generator().manual_seed(1))
        w[32 : 32 + len(values)] = torch.tensor(values)
        w = w.to(wdtype)
        for eps in (0.0, 1e-6):
            y = torch.empty((M, K), dtype=torch.bfloat16, device=d)
            slab, h = mx().mx_rmsnorm_slab(x.to(d), w.to(d), residual=r.to(d), eps=eps, act=act, y=y)
            check(x, r, w, eps, act, slab, h, y, f"{values} eps={eps}")


@pytest.mark.parametrize("act", ["fp8", "fp4"])
@pytest.mark.parametrize("M", [40, 2100])
def test_graph_replays_match_eager(M, act):
    """Two graphs that update their residual in place, replayed in turn."""
    print(f"norm graph M={M} {act}", flush=True)
    d = dev()
    K = 448
    w = (1 + 0.1 * torch.randn((K,), generator=torch.Generator().manual_seed(1))).to(d)
    ins = [(synth.make_activation(M, K, seed=s).to(d), synth.make_activation(M, K, seed=s + 7).float().to(d))
           for s in range(3)]
    want = [mx().mx_rmsnorm_slab(x, w, residual=r, act=act) for x, r in ins]
    graphs = []
    for _ in range(2):
        x, r = (t.clone() for t in ins[0])
        slab, _ = mx().mx_rmsnorm_slab(x, w, residual=r, act=act)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            mx().mx_rmsnorm_slab(x, w, residual=r, residual_out=r, act=act, out=slab)
        graphs.append((g, x, r, slab))
    for turn in range(6):
        g, x, r, slab = graphs[turn % 2]
        k = (2 * turn + 1) % 3
        x.copy_(ins[k][0])
        r.copy_(ins[k][1])
        slab.q.fill_(0xA5)
        slab.s.fill_(0xA5)
        g.replay()
        mx().mx_rmsnorm_slab(ins[turn % 3][0], w, act=act)  # eager work between replays
        torch.cuda.synchronize()
        ref, h = want[k]
        assert torch.equal(slab.q, ref.q) and torch.equal(slab.s, ref.s) and torch.equal(bits(r), bits(h)), turn
    del graphs


@pytest.mark.parametrize("M", [40, 2100])
def test_two_streams_at_once(M):
    print(f"norm two streams M={M}", flush=True)
    d = dev()
    K = 1984
    xs = [synth.make_activation(M, K, seed=s).to(d) for s in (4, 5)]
    want = [mx().mx_rmsnorm_slab(x)[0] for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(mx().mx_rmsnorm_slab(xs[i])[0])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(s.q, want[i].q) and torch.equal(s.s, want[i].s) for s in got[i])
