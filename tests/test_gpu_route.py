"""mx_route against the formula in float64 (oracle.route_ref): ids equal, weights
within 2^-23 (their f32 rounding is 2^-24; the f64 arithmetic before it is off by far
less). An unnormalised softmax without a bias sums its terms in f32: a term exp(-x) is
off by x 2^-23 of itself, and x exp(-x) <= 0.37, so E terms move a sum >= 1 by at most
min(E 0.37, ln E + 1) 2^-23, and its at most 16 + 6 additions by 22 2^-24: 2^-18."""

import numpy as np
import pytest
import torch

import oracle
from helpers import dev, f64, mx

pytestmark = pytest.mark.gpu


def logits(T, E, dtype, seed, ties=False):
    g = torch.Generator().manual_seed(seed)
    l = 2.0 * torch.randn((T, E), generator=g)
    if ties:
        l = l.round()
    return l.to(dtype)


def check(l, k, got=None, **kw):
    ids, w = mx().mx_route(l.to(dev()), k, **{**kw, "bias": None if kw.get("bias") is None else kw["bias"].to(dev())}) \
        if got is None else got
    ref = {**kw, "bias": None if kw.get("bias") is None else f64(kw["bias"])}
    rid, rw = oracle.route_ref(f64(l), k, **ref)
    assert np.array_equal(ids.cpu().numpy(), rid), "ids"
    w = f64(w)
    rel = 2.0**-18 if kw.get("scores", "softmax") == "softmax" and not kw.get("renorm", True) and ref["bias"] is None else 2.0**-23
    assert (np.abs(w - rw) <= rel * np.abs(rw) + 2.0**-149).all(), np.abs(w - rw).max()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,k", [(1, 1), (2, 2), (5, 3), (16, 8), (17, 17), (64, 6), (65, 8), (100, 64), (128, 8),
                                 (130, 1), (256, 8), (257, 8), (300, 10), (512, 64), (515, 4), (1024, 8)])
def test_sizes(E, k, scores, dtype):
    print(f"route E={E} k={k} {scores} {dtype}", flush=True)
    for T in (1, 7, 70):
        for bias in (None, 0.1 * torch.randn(E, generator=torch.Generator().manual_seed(E))):
            check(logits(T, E, dtype, E + T), k, scores=scores, bias=bias, renorm=T != 7, scale=2.5 if T == 70 else 1.0)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top,k", [(8, 8, 3, 3), (12, 3, 2, 8), (16, 2, 1, 8), (64, 8, 3, 6), (64, 64, 20, 20),
                                            (96, 8, 4, 8), (128, 8, 4, 8), (128, 2, 1, 64), (128, 1, 1, 4), (168, 8, 1, 21),
                                            (256, 8, 4, 8), (256, 16, 5, 8), (256, 4, 3, 8), (256, 32, 32, 9),
                                            (320, 5, 2, 8), (512, 8, 4, 8), (512, 64, 7, 8), (1024, 16, 3, 8), (1000, 50, 9, 30)])
def test_groups(E, groups, top, k, scores):
    print(f"route E={E} groups={groups}/{top} k={k} {scores}", flush=True)
    bias = 0.3 * torch.randn(E, generator=torch.Generator().manual_seed(E))
    for b in (None, bias):
        for ties in (False, True):
            check(logits(37, E, torch.float32, E + groups, ties), k, scores=scores, bias=b, groups=groups, top_groups=top)


@pytest.mark.parametrize("E,groups,top", [(24, 1, 1), (24, 4, 2), (256, 8, 2), (300, 1, 1), (300, 3, 2)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_ties_go_to_the_lower_index(E, groups, top, with_bias):
    l = torch.zeros((5, E))
    l[1] = -0.0
    l[2, ::2] = -0.0
    l[3, E // 2:] = 1.0
    l[4] = torch.arange(E) % 3
    check(l, min(6, top * E // groups), scores="sigmoid", bias=torch.zeros(E) if with_bias else None, groups=groups,
          top_groups=top)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,top", [(20, 1, 1), (20, 5, 2), (128, 8, 4), (400, 4, 2)])
@pytest.mark.parametrize("with_bias", [False, True])
def test_masks_infinities_and_nan(E, groups, top, scores, with_bias):
    g = torch.Generator().manual_seed(E)
    l = torch.randn((12, E), generator=g)
    inf, nan = float("inf"), float("nan")
    l[0] = -inf  # nothing left
    l[1] = nan
    l[2] = -inf
    l[2, E - 1] = 0.5  # one left
    l[3, torch.rand(E, generator=g) < 0.7] = -inf
    l[4, torch.rand(E, generator=g) < 0.3] = nan
    l[5, 3] = inf
    l[6, 1::2] = inf
    l[7] = torch.finfo(torch.float32).min  # a mask of the lowest value
    l[8, : E // 2] = torch.finfo(torch.float32).min
    l[9] *= 1e4  # saturated scores
    l[10] *= 1e-30
    l[11] = torch.finfo(torch.float32).max
    b = None
    if with_bias:
        b = 0.1 * torch.randn(E, generator=g)
        b[2], b[E - 2], b[4] = -inf, inf, nan
    check(l, 4, scores=scores, bias=b, groups=groups, top_groups=top)
    check(l, 4, scores=scores, bias=b, groups=groups, top_groups=top, renorm=False)


def test_strided_rows_and_given_outputs():
    d = dev()
    wide = logits(33, 100, torch.float32, 5).to(d)
    for cols, dt in ((slice(4, 68), torch.float32), (slice(3, 67), torch.float32), (slice(8, 72), torch.bfloat16)):
        l = wide.to(dt)[:, cols]
        ids = torch.full((33, 6), -7, dtype=torch.int32, device=d)
        w = torch.full((33, 6), float("nan"), device=d)
        got = mx().mx_route(l, 6, ids=ids, weights=w)
        assert got[0] is ids and got[1] is w
        check(l.cpu(), 6, got=got)


def test_many_tokens_and_none():
    l = logits(100001, 8, torch.float32, 3)
    ids, w = mx().mx_route(l.to(dev()), 2)
    v, i = torch.sort(l, dim=1, descending=True, stable=True)
    assert torch.equal(ids.cpu().long(), i[:, :2])
    assert (w.cpu() - torch.softmax(v[:, :2].double(), 1)).abs().max() <= 2.0**-23
    ids, w = mx().mx_route(l[:0].to(dev()), 2)
    assert ids.shape == (0, 2) and w.shape == (0, 2)


def test_graph_and_other_stream():
    d = dev()
    ins = [logits(300, 128, torch.float32, s).to(d) for s in (1, 2, 3)]
    b = (0.1 * torch.randn(128, generator=torch.Generator().manual_seed(9))).to(d)
    x = ins[0].clone()
    ids, w = mx().mx_route(x, 8, scores="sigmoid", bias=b, groups=8, top_groups=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        i2, w2 = mx().mx_route(x, 8, scores="sigmoid", bias=b, groups=8, top_groups=4)
    torch.cuda.synchronize()
    assert torch.equal(ids, i2) and torch.equal(w, w2)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mx().mx_route(x, 8, scores="sigmoid", bias=b, groups=8, top_groups=4, ids=ids, weights=w)
    for xin in ins + ins[:1]:
        x.copy_(xin)
        g.replay()
        torch.cuda.synchronize()
        e = mx().mx_route(xin, 8, scores="sigmoid", bias=b, groups=8, top_groups=4)
        assert torch.equal(ids, e[0]) and torch.equal(w, e[1])
    del g
