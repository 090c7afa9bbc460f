"""mx_block_norm_slab against the formula in float64.

h: its terms are off by fewer than 16 roundings of 2^-24 of them before h is rounded
(the residual's product 1; the post norm's sum of squares 8 2^-24 halved by the root,
its rstd, the products with rstd, weight and gate, the addition: 10), so the stored h
lies between the roundings of the ends of that range. y: likewise from the stored h,
within the bound that oracle.block_y_ref derives. Codes and scales are the exact
quantization of the y that the same call wrote."""

import numpy as np
import pytest
import torch

import oracle
import synth
from helpers import dev, f64, mx, u8

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32


def rounded(v, dt):
    if dt == BF16:
        return oracle.bf16_round(np.asarray(v, np.float64).astype(np.float32).astype(np.float64))
    with np.errstate(over="ignore"):
        return np.asarray(v, np.float64).astype(np.float32).astype(np.float64)


def between(got, v, err, dt, what):
    """got lies between the roundings of v - err and v + err (NaN where v is NaN)."""
    with np.errstate(invalid="ignore", over="ignore"):
        lo, hi = rounded(v - err, dt), rounded(v + err, dt)
        nan = np.isnan(v)
        assert np.array_equal(np.isnan(got), nan), f"{what}: NaN pattern"
        ok = (got >= lo) & (got <= hi) | nan | (np.isinf(v) & (got == v))
        assert ok.all(), f"{what}: {int((~ok).sum())} of {ok.size} outside, first at {np.argwhere(~ok)[0]}: {got[~ok][0]} not in [{lo[~ok][0]}, {hi[~ok][0]}]"


def slab_of(y, act):
    if act == "fp4":
        return oracle.fp4_slab(*oracle.quantize_fp4(y))
    codes, scales = oracle.quantize_mx(y)
    M, K = y.shape
    R = (M + 255) // 256 * 256
    q, s = np.zeros((K // 64, R, 64), np.uint8), np.zeros((K // 64, R, 2), np.uint8)
    q[:, :M] = codes.reshape(M, -1, 64).transpose(1, 0, 2)
    s[:, :M] = scales.reshape(M, -1, 2).transpose(1, 0, 2)
    return q, s


def rows_of(v, M):
    v = f64(v)
    v = v[None] if v.ndim == 1 else v
    return np.repeat(v, M // v.shape[0], axis=0)


def check(x, r, got, y, rows=None, act="fp8", eps=1e-6, alpha=1.0, post=False, pw=None, gate=None, kind="rms", w=None,
          scale=None, shift=None):
    M = x.shape[0]
    sel = slice(None) if rows is None else rows
    pick = lambda v: None if v is None else rows_of(v, M)[sel if rows is None else rows.numpy()]  # noqa: E731
    one = lambda v: None if v is None else f64(v)  # noqa: E731
    slab, h = got
    hv, mag = oracle.block_h_ref(f64(x[sel]), f64(r[sel]), alpha, post, one(pw), pick(gate), eps)
    hg, yg = f64(h[sel]), f64(y[sel])
    between(hg, hv, mag * 2.0**-20, r.dtype, "h")
    yv, err = oracle.block_y_ref(hg, kind, one(w), pick(scale), pick(shift), eps)
    between(yg, yv, err, BF16, "y")
    if act is not None and rows is None:
        q, s = slab_of(f64(y), act)
        assert np.array_equal(u8(slab.s), s) and np.array_equal(u8(slab.q), q), "slab"


def make(M, K, rdt, vdt, seed, post, gate, mod, weight=True):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    d = {"x": synth.make_activation(M, K, seed=seed), "r": (3.0 * rn(M, K)).to(rdt)}
    d["pw"] = (1 + 0.2 * rn(K)).to(vdt) if post else None
    d["gate"] = None if gate is None else (0.5 + 0.2 * rn(gate, K)).to(vdt) if gate else (0.5 + 0.2 * rn(K)).to(vdt)
    d["w"] = (1 + 0.2 * rn(K)).to(vdt) if weight else None
    d["scale"] = None if mod is None else (0.3 * rn(mod, K)).to(vdt)
    d["shift"] = None if mod is None else (0.3 * rn(mod, K)).to(vdt)
    return d


def call(d, act="fp8", kind="rms", post=False, alpha=1.0, eps=1e-6, **kw):
    v = {k: None if t is None else t.to(dev()) for k, t in d.items()}
    y = torch.empty(v["x"].shape, dtype=BF16, device=dev())
    got = mx().mx_block_norm_slab(v["x"], v["r"], post=post, post_weight=v["pw"], gate=v["gate"], residual_scale=alpha,
                                  kind=kind, weight=v["w"], scale=v["scale"], shift=v["shift"], eps=eps, act=act, y=y, **kw)
    return got, y


def run(M, K, rdt, vdt, act="fp8", kind="rms", post=False, gate=None, mod=None, alpha=1.0, eps=1e-6, rows=None, seed=0,
        weight=True):
    print(f"block norm {M}x{K} {rdt} {vdt} {act} {kind} post={post} gate={gate} mod={mod}", flush=True)
    d = make(M, K, rdt, vdt, seed + M + K, post, gate, mod, weight)
    got, y = call(d, act, kind, post, alpha, eps)
    check(got=got, y=y, rows=rows, act=act, eps=eps, alpha=alpha, post=post, kind=kind, **d)
    return d, got, y


SHAPES = [(1, 64), (3, 192), (17, 4096), (257, 576), (6, 5120), (4, 8256), (2, 16448), (2, 65536)]


@pytest.mark.parametrize("act", ["fp8", "fp4"])
@pytest.mark.parametrize("rdt", [BF16, F32])
@pytest.mark.parametrize("M,K", SHAPES)
def test_row_form(M, K, rdt, act):
    run(M, K, rdt, BF16, act, post=True, gate=0, alpha=0.75)
    run(M, K, rdt, F32, act, kind="layer", gate=M, mod=1)


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("vdt", [BF16, F32])
@pytest.mark.parametrize("post,gate,mod,weight", [(False, None, None, False), (True, None, None, True), (True, 1, None, True),
                                                  (False, 3, 2, True), (True, 6, 6, False), (True, 0, 3, True)])
def test_options(post, gate, mod, weight, vdt, kind):
    run(6, 320, BF16, vdt, kind=kind, post=post, gate=gate, mod=mod, weight=weight, alpha=1.5)


@pytest.mark.parametrize("K", [32, 96, 160, 4128])
def test_fp4_and_no_slab_take_any_multiple_of_32(K):
    run(19, K, BF16, F32, "fp4", kind="layer", post=True, gate=1, mod=19)
    d, got, y = run(19, K, BF16, F32, None, kind="layer", post=True, gate=1, mod=19)
    assert got[0] is y
    z, h = mx().mx_block_norm_slab(*(d[n].to(dev()) for n in ("x", "r")), act=None)
    assert z.shape == (19, K) and z.dtype == BF16


@pytest.mark.parametrize("M,K,rdt", [(2049, 2048, BF16), (2050, 1088, F32), (32769, 2112, BF16), (32770, 4096, F32),
                                     (32768, 5120, BF16), (32769, 5120, F32), (32769, 8192, BF16)])
@pytest.mark.parametrize("act", ["fp8", "fp4"])
def test_tile_form(M, K, rdt, act):
    print(f"block norm {M}x{K} {rdt} {act}", flush=True)
    rows = np.unique(np.concatenate([np.arange(9), np.random.default_rng(M).integers(0, M, 60), np.arange(M - 9, M)]))
    n, post = 2 if M % 2 == 0 else 1, act == "fp4"
    d = make(2, K, rdt, F32 if act == "fp8" else BF16, M, post, n, n)
    g = torch.Generator(device=dev()).manual_seed(M)  # the large operands are drawn there
    d["x"] = torch.randn((M, K), generator=g, device=dev()).to(BF16)
    d["r"] = (3.0 * torch.randn((M, K), generator=g, device=dev())).to(rdt)
    got, y = call(d, act, "layer", post)
    check(got=got, y=y, rows=torch.from_numpy(rows), act=act, kind="layer", post=post, **d)
    # The slab is that of the quantizer on y, padded rows included.
    quant = mx().mx_quantize_act_slab if act == "fp8" else mx().mx_fp4_quantize_act_slab
    ref = quant(y)
    assert torch.equal(ref.q, got[0].q) and torch.equal(ref.s, got[0].s)


def test_equals_the_residual_rms_norm_where_both_apply():
    # h is the same rounded f32 sum; y may differ by a rounding, as both are within their bounds.
    d = make(33, 1024, BF16, BF16, 7, False, None, None)
    got, y = call(d)
    slab, h = mx().mx_rmsnorm_slab(d["x"].to(dev()), d["w"].to(dev()), residual=d["r"].to(dev()))
    assert torch.equal(h, got[1])
    assert (slab.q != got[0].q).float().mean() < 1e-4


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("mag", [1e30, 1e19, 1e-22, 1e-32])
def test_magnitudes_past_the_squares_range(mag, kind):
    # The squares leave f32's range; eps = 0 hides nothing.
    g = torch.Generator().manual_seed(1)
    d = {n: None for n in ("pw", "gate", "w", "scale", "shift")}
    d["r"] = torch.randn((5, 640), generator=g) * mag
    d["x"] = (torch.randn((5, 640), generator=g) * mag).to(BF16)
    for post in (False, True):
        if post:
            d["r"] = torch.randn((5, 640), generator=g)
        got, y = call(d, kind=kind, eps=0.0, post=post)
        check(got=got, y=y, eps=0.0, kind=kind, post=post, **d)


def test_mean_far_from_zero():
    d = make(9, 2048, F32, F32, 3, False, None, None)
    d["r"] += 1000.0
    got, y = call(d, kind="layer")
    check(got=got, y=y, kind="layer", **d)


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_zero_infinite_and_nan_rows(kind):
    d = make(8, 256, BF16, F32, 11, True, None, None)
    d["x"][0] = d["r"][0] = 0.0
    d["x"][1] = 0.0  # the post norm of zeros
    d["r"][2, 7] = float("nan")
    d["x"][3, 9] = float("nan")
    d["r"][4, 100] = float("inf")
    d["x"][5, 200] = float("-inf")
    got, y = call(d, kind=kind, post=True)
    check(got=got, y=y, kind=kind, post=True, **d)


def test_in_place_residual_strides_and_padding():
    d = dev()
    M, K = 21, 448
    src = make(M, K, BF16, F32, 5, True, 3, 7)
    want, wy = call(src, kind="layer", post=True)
    wide = {n: torch.full((M + 2, K + 64), 9.0, dtype=src[n].dtype, device=d) for n in ("x", "r")}
    for n, t in wide.items():
        t[1 : M + 1, 32 : K + 32] = src[n].to(d)
    x, r = (wide[n][1 : M + 1, 32 : K + 32] for n in ("x", "r"))
    mods = torch.zeros((7, 3, K), device=d)  # scale and shift as rows of one tensor
    mods[:, 1], mods[:, 2] = src["scale"].to(d), src["shift"].to(d)
    slab, h = mx().mx_block_norm_slab(x, r, post=True, post_weight=src["pw"].to(d), gate=src["gate"].to(d), kind="layer",
                                      weight=src["w"].to(d), scale=mods[:, 1], shift=mods[:, 2], residual_out=r)
    assert h is r and torch.equal(h, want[1]) and torch.equal(slab.q, want[0].q) and torch.equal(slab.s, want[0].s)
    edge = wide["r"].clone()
    edge[1 : M + 1, 32 : K + 32] = 9.0
    assert (edge == 9.0).all()


def test_graph_and_other_stream():
    d = dev()
    ins = [make(300, 512, BF16, F32, s, True, 2, 2) for s in (1, 2, 3)]
    v = {n: t.to(d) for n, t in ins[0].items()}
    y = torch.empty((300, 512), dtype=BF16, device=d)

    def step(out=None, ro=None):
        return mx().mx_block_norm_slab(v["x"], v["r"], post=True, post_weight=v["pw"], gate=v["gate"], kind="layer",
                                       weight=v["w"], scale=v["scale"], shift=v["shift"], out=out, residual_out=ro, y=y)

    slab, h = step()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step(slab, h)
    side = torch.cuda.Stream()
    for src in ins + ins[:1]:
        for n in v:
            v[n].copy_(src[n])
        g.replay()
        torch.cuda.synchronize()
        a = [t.clone() for t in (slab.q, slab.s, h, y)]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            s2, h2 = step()
        torch.cuda.synchronize()
        for p, q in zip(a, (s2.q, s2.s, h2, y)):
            assert torch.equal(p, q)
    del g
