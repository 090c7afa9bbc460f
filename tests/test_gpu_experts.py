"""mx_fp4_experts against the formula in float64 (oracle.experts_ref, which derives
its bound), on each of its kernels: a few tokens, tiles of 128 weight rows, tiles of 256
for experts with many pairs."""

import numpy as np
import pytest
import torch

import oracle
import synth
from helpers import dev, f64, mx

pytestmark = pytest.mark.gpu


def weights(E, N, K, seed):
    g = torch.Generator().manual_seed(seed)
    w = 2.0 * torch.randn((E, N, K), generator=g) / K**0.5
    return mx().mx_fp4_quantize_experts(w.to(dev())), w


def values(w):
    return oracle.dequantize_fp4(*oracle.quantize_fp4(f64(w)))


def route(T, k, E, seed, skew=0.0):
    g = torch.Generator().manual_seed(seed)
    l = torch.randn((T, E), generator=g) + skew * torch.randn((1, E), generator=g)
    v, i = l.sort(dim=1, descending=True)
    return i[:, :k].to(torch.int32).contiguous(), torch.softmax(v[:, :k], dim=1).contiguous()


def make(T, k, E, H, I, seed=0, skew=0.0):
    x = synth.make_activation(T, H, seed=seed + 1)
    ids, w = route(T, k, E, seed + 2, skew)
    up, uw = weights(E, 2 * I, H, seed + 3)
    down, dw = weights(E, H, I, seed + 4)
    return x, ids, w, up, down, values(uw), values(dw)


def run(x, ids, w, up, down, **kw):
    d = dev()
    return mx().mx_fp4_experts(x.to(d), ids.to(d), w.to(d), up, down, **kw)


def close(y, x, ids, w, uv, dv, act, gate="silu"):
    ref, tol = oracle.experts_ref(f64(x), ids.numpy(), f64(w), uv, dv, act, gate)
    err = np.abs(f64(y) - ref)
    assert (err <= tol).all(), f"{int((err > tol).sum())} of {err.size}, worst {np.nanmax(err / tol)}, NaN {np.isnan(err).sum()}"


# T, k, E, H, I: a few tokens; tiles of 128; tiles of 256 (64 pairs an expert and more).
FEW = [(1, 1, 1, 32, 32), (1, 8, 16, 256, 96), (2, 3, 3, 96, 160), (13, 3, 5, 160, 64), (16, 8, 8, 128, 32), (16, 1, 40, 608, 352),
       (2, 64, 70, 64, 32), (5, 4, 6, 1056, 416)]
SMALL = [(17, 1, 3, 96, 160), (17, 8, 20, 32, 32), (40, 4, 8, 544, 288), (130, 2, 5, 64, 32), (100, 1, 2, 1120, 96), (3, 50, 60, 288, 128),
         (200, 5, 17, 1184, 416)]
LARGE = [(64, 1, 1, 32, 32), (129, 1, 2, 128, 64), (130, 1, 1, 160, 128), (300, 2, 3, 608, 352), (513, 1, 4, 1152, 384),
         (260, 4, 2, 96, 416), (1500, 3, 7, 288, 160), (700, 1, 1, 544, 288)]


@pytest.mark.parametrize("act", ["fp8", "fp4"])
@pytest.mark.parametrize("T,k,E,H,I", FEW + SMALL + LARGE)
def test_against_the_formula(T, k, E, H, I, act):
    print(f"experts T={T} k={k} E={E} H={H} I={I} {act}", flush=True)
    k = min(k, E)
    x, ids, w, up, down, uv, dv = make(T, k, E, H, I, seed=T + H)
    gate = "gelu" if I % 64 else "silu"
    y = run(x, ids, w, up, down, act=act, gate=gate)
    assert y.shape == (T, H) and y.dtype == torch.bfloat16
    close(y, x, ids, w, uv, dv, act, gate)


@pytest.mark.parametrize("act", ["fp8", "fp4"])
@pytest.mark.parametrize("T,E", [(11, 5), (50, 5), (400, 5)])
def test_one_expert_takes_all_and_others_none(T, E, act):
    x, _, w, up, down, uv, dv = make(T, 2, E, 160, 96, seed=3)
    ids = torch.full((T, 2), 3, dtype=torch.int32)
    ids[:, 1] = torch.arange(T) % 2  # experts 2 and 4 have no token
    close(run(x, ids, w, up, down, act=act), x, ids, w, uv, dv, act)


@pytest.mark.parametrize("T", [9, 60, 500])
def test_skipped_and_repeated_pairs(T):
    x, ids, w, up, down, uv, dv = make(T, 4, 6, 96, 64, seed=5)
    ids[0] = torch.tensor([-1, 6, 2**31 - 1, -(2**31)])  # none of them an expert
    w[0] = float("nan")  # and their weights do not count
    ids[1] = 2  # four times the same
    ids[2] = torch.tensor([4, 1, 4, -5])
    ids[3, 1] = 100
    w[3, 1] = float("inf")
    ids[4:, 3] = ids[4:, 0]
    y = run(x, ids, w, up, down)
    assert not y[0].any()
    wz = torch.where((ids >= 0) & (ids < 6), w, torch.zeros_like(w))
    close(y, x, ids, wz, uv, dv, "fp8")


@pytest.mark.parametrize("T", [7, 100, 600])
@pytest.mark.parametrize("act", ["fp8", "fp4"])
def test_special_rows_stay_to_themselves(T, act):
    x, ids, w, up, down, _, _ = make(T, 2, 4, 160, 64, seed=7)
    y0 = run(x, ids, w, up, down, act=act)
    z = x.clone()
    z[2, 5], z[4, 100], z[T - 1, 0] = float("nan"), float("inf"), float("-inf")
    z[3] = 0.0
    wz = w.clone()
    wz[5, 1] = float("nan")
    y = run(z, ids, wz, up, down, act=act)
    assert torch.isnan(y[[2, 4, 5, T - 1]]).all() and not y[3].any()
    rest = [t for t in range(T) if t not in (2, 3, 4, 5, T - 1)]
    assert torch.equal(y[rest], y0[rest])


def test_every_kernel_gives_the_same_where_sums_are_exact():
    # One nonzero weight a row: every sum has one term, so the three kernels (taken by T)
    # must agree bit for bit, row by row, whichever tile or lane a row falls into.
    E, H, I, d = 3, 416, 352, dev()
    g = torch.Generator().manual_seed(1)

    def pick(N, K, seed):
        w = torch.zeros((E, N, K))
        col = torch.randint(0, K, (E, N), generator=torch.Generator().manual_seed(seed))
        w.scatter_(2, col[..., None], torch.where(torch.rand((E, N, 1), generator=g) < 0.5, -1.0, 2.0))
        return mx().mx_fp4_quantize_experts(w.to(d))

    up, down = pick(2 * I, H, 2), pick(H, I, 3)
    x = synth.make_activation(700, H, seed=4)
    ids = torch.randint(0, E, (700, 1), generator=g).to(torch.int32)
    w = torch.rand((700, 1), generator=g)
    for act in ("fp8", "fp4"):
        large = run(x, ids, w, up, down, act=act)
        for T, step in ((16, 16), (100, 100), (1, 37)):
            for t in range(0, 700 - T, step):
                assert torch.equal(run(x[t : t + T], ids[t : t + T], w[t : t + T], up, down, act=act), large[t : t + T]), (act, T, t)
                if T == 1 and t > 300:
                    break


def test_strided_rows_given_output_and_workspace():
    d = dev()
    for T in (5, 90, 400):
        x, ids, w, up, down, _, _ = make(T, 2, 4, 96, 64, seed=9)
        want = run(x, ids, w, up, down)
        wide = torch.full((T, 160), float("nan"), dtype=torch.bfloat16, device=d)
        wide[:, 32:128] = x.to(d)
        need = mx().mx_fp4_experts_ws_bytes(T, 2, 4, 96, 64)
        pool = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device=d)  # NaN scales, should any be read
        y = torch.full((T + 2, 96), 7.0, dtype=torch.bfloat16, device=d)
        got = mx().mx_fp4_experts(wide[:, 32:128], ids.to(d), w.to(d), up, down, y=y[1 : T + 1], workspace=pool[256 : 256 + need])
        assert torch.equal(got, want)
        assert (y[0] == 7.0).all() and (y[T + 1] == 7.0).all()
        assert (pool[:256] == 0xFF).all() and (pool[256 + need :] == 0xFF).all()


def test_many_pairs_many_experts_and_none():
    # Several chunks of the plan; 1024 experts; no token.
    x, ids, w, up, down, uv, dv = make(3001, 3, 7, 64, 32, seed=11, skew=1.0)
    close(run(x, ids, w, up, down, act="fp4"), x, ids, w, uv, dv, "fp4")
    x, ids, w, up, down, uv, dv = make(300, 64, 1024, 32, 32, seed=12)
    close(run(x, ids, w, up, down, act="fp4"), x, ids, w, uv, dv, "fp4")
    assert run(x[:0], ids[:0], w[:0], up, down).shape == (0, 32)


def test_experts_past_4_gib():
    # up: 300 experts of 8192 x 4096, 4.7 GiB of codes. The last expert's result is that of
    # the same slabs alone.
    E, H, I, d = 300, 4096, 4096, dev()
    g = torch.Generator(device=d).manual_seed(2)

    def big(N, K):
        sq, ss = ((K + 127) // 128, N // 16, 4, 16, 16), ((K + 127) // 128, N, 4)
        q = torch.empty((E,) + sq, dtype=torch.uint8, device=d)
        for e in range(E):
            q[e] = torch.randint(0, 256, sq, generator=g, device=d, dtype=torch.uint8)
        return mx().FP4Experts(q, torch.full((E,) + ss, 120, dtype=torch.uint8, device=d), N, K)

    up, down = big(2 * I, H), big(H, I)
    assert up.q.numel() > 1 << 32
    last = [mx().FP4Experts(t.q[E - 1 :].contiguous(), t.s[E - 1 :].contiguous(), t.rows, t.K) for t in (up, down)]
    for T in (3, 20, 100):
        x = synth.make_activation(T, H, seed=T).to(d)
        w = torch.ones((T, 1), device=d)
        # (A tile's kernel goes with the pairs an expert: 100 of one, or of 300.)
        for act in ("fp8", "fp4"):
            y = mx().mx_fp4_experts(x, torch.full((T, 1), E - 1, dtype=torch.int32, device=d), w, up, down, act=act)
            z = mx().mx_fp4_experts(x, torch.zeros((T, 1), dtype=torch.int32, device=d), w, *last, act=act)
            if T < 64:
                assert torch.equal(y, z)
            else:
                assert ((y.float() - z.float()).norm() / z.float().norm()).item() < 2.0**-6


def test_quantize_experts_is_the_slab_quantizer():
    w = torch.randn((3, 40, 160), generator=torch.Generator().manual_seed(1)).to(dev())
    ex = mx().mx_fp4_quantize_experts(w)
    for e in range(3):
        s = mx().mx_fp4_quantize_weight_slab(w[e])
        assert torch.equal(s.q, ex.q[e]) and torch.equal(s.s, ex.s[e])
    out = mx().mx_fp4_quantize_experts(w.to(torch.bfloat16), out=ex)
    assert out is ex


@pytest.mark.parametrize("T", [6, 80, 500])
def test_graphs_and_two_streams(T):
    d = dev()
    k, E, H, I = 2, 4, 160, 96
    x0, ids0, w0, up, down, _, _ = make(T, k, E, H, I, seed=13)
    cases = [(x0, ids0, w0)]
    for s in (14, 15):
        ids, w = route(T, k, E, s, 2.0)
        cases.append((synth.make_activation(T, H, seed=s), ids, w))
    cases = [tuple(t.to(d) for t in c) for c in cases]
    x, ids, w = (t.clone() for t in cases[0])
    nb = mx().mx_fp4_experts_ws_bytes(T, k, E, H, I)
    ws = [torch.empty((nb,), dtype=torch.uint8, device=d) for _ in range(2)]
    y = torch.empty((T, H), dtype=torch.bfloat16, device=d)
    mx().mx_fp4_experts(x, ids, w, up, down, y=y, workspace=ws[0])
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        mx().mx_fp4_experts(x, ids, w, up, down, y=y, workspace=ws[0])
    want = [mx().mx_fp4_experts(*c, up, down) for c in cases]
    side = torch.cuda.Stream()
    for i in (0, 1, 2, 0, 2):
        for t, s in zip((x, ids, w), cases[i]):
            t.copy_(s)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):  # beside the replay, on a workspace of its own
            z = mx().mx_fp4_experts(*cases[2 - i], up, down, workspace=ws[1])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i]) and torch.equal(z, want[2 - i]), f"case {i}"
    del g


def test_repeats_bit_for_bit():
    x, ids, w, up, down, _, _ = make(2000, 4, 9, 288, 160, seed=17, skew=1.0)
    a = run(x, ids, w, up, down)
    for _ in range(5):
        assert torch.equal(run(x, ids, w, up, down), a)
