"""mx_block_norm_slab's sums and products are float64: h and y are the formula's values,
rounded to f32 and then to their type, but where the float64 value itself is in doubt.

Tolerances: a sum of K <= 65536 terms is off by at most K 2^-53 = 2^-37 of its magnitude,
the few products by 2^-50; so 2^-36 of the terms. Variances of bf16 h as a difference of
sums: the mean's rounding is 2^-53 of the mean square, which is at most 2^16 K times the
variance where values differ at all (K = 65536: 2^-21 of it, 2^-22 of its root)."""

import numpy as np
import pytest
import torch

import oracle
import synth
from helpers import dev, f64, mx
from test_gpu_block_norm import BF16, F32, between, rounded, rows_of

pytestmark = pytest.mark.gpu


def exact(v, err, dt, got, what):
    between(got, v, err, dt, what)  # err so small that it is the rounded value, but for a tie or two
    assert (got != rounded(rounded(v, F32), dt)).mean() < 1e-4, what


def run(M, K, rdt, vdt, kind, post, gate, mod, weight, rows=None, act="fp8"):
    print(f"block norm {M}x{K} {rdt} {vdt} {kind} post={post} gate={gate} mod={mod} weight={weight}", flush=True)
    d = dev()
    g = torch.Generator(device=d).manual_seed(M + K)
    rn = lambda *s: torch.randn(s, generator=g, device=d)  # noqa: E731
    x, r = rn(M, K).to(BF16), (3.0 * rn(M, K)).to(rdt)
    n = 2 if M % 2 == 0 else 1
    vec = lambda on, *s: rn(*s).to(vdt) if on else None  # noqa: E731
    pw, w = vec(post and weight, K), vec(weight, K)
    gt, scale, shift = vec(gate, n, K), vec(mod, n, K), vec(mod, n, K)
    y = torch.empty((M, K), dtype=BF16, device=d)
    slab, h = mx().mx_block_norm_slab(x, r, post=post, post_weight=pw, gate=gt, residual_scale=0.75, kind=kind, weight=w,
                                      scale=scale, shift=shift, act=act, y=y)
    rows = np.arange(M) if rows is None else rows
    sel = torch.from_numpy(rows).to(d)
    pick = lambda v: None if v is None else rows_of(v, M)[rows]  # noqa: E731
    one = lambda v: None if v is None else f64(v)  # noqa: E731
    hv, mag = oracle.block_h_ref(f64(x[sel]), f64(r[sel]), 0.75, post, one(pw), pick(gt))
    hg, yg = f64(h[sel]), f64(y[sel])
    exact(hv, mag * 2.0**-36, rdt, hg, "h")
    yv, _ = oracle.block_y_ref(hg, kind, one(w), pick(scale), pick(shift))
    rstd = 1.0 / np.sqrt(np.mean((hg - (hg.mean(-1, keepdims=True) if kind == "layer" else 0.0)) ** 2, -1, keepdims=True) + 1e-6)
    factor = rstd * np.abs(1.0 if w is None else one(w)) * (1.0 if scale is None else 1.0 + np.abs(pick(scale)))
    terms = factor * (np.abs(hg) + np.abs(hg).mean(-1, keepdims=True)) + (0.0 if shift is None else np.abs(pick(shift)))
    exact(yv, terms * 2.0**-36, BF16, yg, "y")
    quant = mx().mx_quantize_act_slab if act == "fp8" else mx().mx_fp4_quantize_act_slab
    ref = quant(y)
    assert torch.equal(ref.q, slab.q) and torch.equal(ref.s, slab.s)


OPTIONS = [(False, False, False, True), (False, False, True, False), (False, True, False, True), (False, True, True, True),
           (True, False, False, True), (True, True, True, False)]


@pytest.mark.parametrize("post,gate,mod,weight", OPTIONS)
@pytest.mark.parametrize("M,K,rdt,vdt", [(6, 5120, BF16, F32), (7, 1088, F32, BF16), (2050, 1088, BF16, BF16),
                                         (2049, 2048, F32, F32)])
def test_few_and_short_rows(M, K, rdt, vdt, post, gate, mod, weight):
    for kind in ("rms", "layer"):
        run(M, K, rdt, vdt, kind, post, gate, mod, weight, rows=np.unique(np.r_[np.arange(3), M // 2, np.arange(M - 3, M)]),
            act="fp8" if gate else "fp4")


@pytest.mark.parametrize("post,gate,mod,weight", OPTIONS)
@pytest.mark.parametrize("M,K", [(32769, 4096), (32770, 4160)])
def test_long_rows_in_tiles(M, K, post, gate, mod, weight):
    rows = np.unique(np.r_[np.arange(9), np.random.default_rng(K).integers(0, M, 30), np.arange(M - 9, M)])
    run(M, K, BF16, F32 if mod else BF16, "layer" if mod else "rms", post, gate, mod, weight, rows, "fp4" if gate else "fp8")


@pytest.mark.parametrize("M,K", [(5, 64), (5, 5120), (2, 65536), (2051, 2048)])
def test_variance_of_nearly_equal_bf16_values(M, K):
    # All values 256 but one, by one bf16 step; and all the same: exactly 0.
    d = dev()
    r = torch.full((M, K), 256.0, dtype=BF16)
    r[1:, K - 3] = 258.0
    y = torch.empty((M, K), dtype=BF16, device=d)
    for eps in (0.0, 1e-6):
        mx().mx_block_norm_slab(torch.zeros((M, K), dtype=BF16, device=d), r.to(d), kind="layer", eps=eps, y=y)
        got = f64(y)
        h = f64(r)
        diff = h - h.mean(-1, keepdims=True)
        with np.errstate(invalid="ignore", divide="ignore"):
            want = diff / np.sqrt((diff * diff).mean(-1, keepdims=True) + eps)
        between(got[1:], want[1:], np.abs(want[1:]) * 2.0**-21, BF16, "y")
        assert np.isnan(got[0]).all() if eps == 0.0 else (got[0] == 0.0).all()


def test_variance_of_bf16_values_far_from_zero():
    d = dev()
    g = torch.Generator().manual_seed(4)
    r = (1000.0 + 4.0 * torch.randn((9, 4096), generator=g)).to(BF16)
    y = torch.empty((9, 4096), dtype=BF16, device=d)
    mx().mx_block_norm_slab(synth.make_activation(9, 4096, seed=1).to(d) * 0, r.to(d), kind="layer", y=y)
    want, _ = oracle.block_y_ref(f64(r), "layer")
    # The mean square is 2^16 times the variance: 2^-53 2^16, and the sums' 2^-41 of it.
    between(f64(y), want, np.abs(want) * 2.0**-24 + 2.0**-36, BF16, "y")
