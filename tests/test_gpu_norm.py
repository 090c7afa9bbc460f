"""GPU parity of mx_rmsnorm_slab against the oracle's formula in float64.

The kernel computes the mean square and the product in float64 and rounds
through f32 to bf16, as the oracle does; the float64 sums are associated
differently, which moves a value by at most about K 2^-53 of itself and so
changes a rounding with a probability below 2^-20 per element: h, y, codes and
scales are compared bit for bit."""

import numpy as np
import pytest
import torch

import oracle
import synth
from helpers import dev, f64, mx, u8

pytestmark = pytest.mark.gpu


def bits(t):
    return t.cpu().view(torch.int16 if t.dtype == torch.bfloat16 else torch.int32)


def inputs(M, K, res, gain, seed):
    g = torch.Generator().manual_seed(seed)
    x = synth.make_activation(M, K, seed=seed)
    r = None
    if res is not None:
        r = (3.0 * torch.randn((M, K), generator=g)).to(res)
    w = None
    if gain is not None:
        w = (1.0 + 0.2 * torch.randn((K,), generator=g)).to(gain)
    return x, r, w


def reference(x, r, w, eps, act):
    h, y = oracle.rmsnorm_ref(f64(x), None if r is None else f64(r), None if w is None else f64(w), eps,
                              residual_f32=r is not None and r.dtype == torch.float32)
    if act == "fp4":
        return h, y, oracle.fp4_slab(*oracle.quantize_fp4(y))
    codes, scales = oracle.quantize_mx(y)
    M, K = y.shape
    R = (M + 255) // 256 * 256
    q, s = np.zeros((K // 64, R, 64), np.uint8), np.zeros((K // 64, R, 2), np.uint8)
    q[:, :M] = codes.reshape(M, -1, 64).transpose(1, 0, 2)
    s[:, :M] = scales.reshape(M, -1, 2).transpose(1, 0, 2)
    return h, y, (q, s)


def check(x, r, w, eps, act, slab, h, y, what):
    rh, ry, (q, s) = reference(x, r, w, eps, act)
    if r is not None:
        assert np.array_equal(f64(h), rh, equal_nan=True), f"{what}: h"
    if y is not None:
        assert np.array_equal(f64(y), ry, equal_nan=True), f"{what}: y"
    assert np.array_equal(u8(slab.s), s), f"{what}: scales"
    assert np.array_equal(u8(slab.q), q), f"{what}: codes"


@pytest.mark.parametrize("act", ["fp8", "fp4"])
@pytest.mark.parametrize("res", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(1, 64), (1, 5120), (3, 192), (17, 4096), (257, 576), (16, 8192), (5, 8256), (2, 16448), (3, 11008), (2, 65536)])
def test_few_rows(M, K, res, act):
    print(f"norm M={M} K={K} res={res} {act}", flush=True)
    d = dev()
    x, r, w = inputs(M, K, res, torch.bfloat16, M + K)
    y = torch.empty((M, K), dtype=torch.bfloat16, device=d)
    slab, h = mx().mx_rmsnorm_slab(x.to(d), w.to(d), residual=None if r is None else r.to(d), act=act, y=y)
    check(x, r, w, 1e-6, act, slab, h, y, f"{M}x{K}")


@pytest.mark.parametrize("K", [32, 96, 160, 4128])
def test_fp4_takes_any_multiple_of_32(K):
    print(f"norm fp4 K={K}", flush=True)
    d = dev()
    x, r, w = inputs(19, K, torch.bfloat16, torch.float32, K)
    slab, h = mx().mx_rmsnorm_slab(x.to(d), w.to(d), residual=r.to(d), act="fp4")
    check(x, r, w, 1e-6, "fp4", slab, h, None, f"K={K}")


@pytest.mark.parametrize("act", ["fp8", "fp4"])
@pytest.mark.parametrize("res", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("K", [192, 2048, 2112, 4096, 5120, 5184, 8192])
def test_many_rows(K, res, act):
    """The tiled form, from 2048 rows or, for K > 2048, 32768 (past it long f32 rows)."""
    M = 4100 if K <= 2048 else 32772
    print(f"norm M={M} K={K} res={res} {act}", flush=True)
    d = dev()
    g = torch.Generator(device=d).manual_seed(K)
    x = torch.randn((M, K), generator=g, device=d).to(torch.bfloat16)
    r = None if res is None else (2 * torch.randn((M, K), generator=g, device=d)).to(res)
    w = (1 + 0.1 * torch.randn((K,), generator=g, device=d)).to(torch.bfloat16)
    y = torch.empty((M, K), dtype=torch.bfloat16, device=d)
    slab, h = mx().mx_rmsnorm_slab(x, w, residual=r, act=act, y=y)
    rows = torch.cat([torch.arange(0, 20), torch.arange(2040, 2056), torch.arange(M - 20, M)])
    R = slab.s.shape[1]
    rd = rows.to(d)
    rh, ry, (q, s) = reference(x[rd].cpu(), None if r is None else r[rd].cpu(), w.cpu(), 1e-6, act)
    if r is not None:
        assert np.array_equal(f64(h[rd]), rh)
    assert np.array_equal(f64(y[rd]), ry)
    assert np.array_equal(u8(slab.s[:, rd]), s[:, : len(rows)])
    # Every row against the quantizer of the y that the same call wrote.
    if act == "fp4":
        ref = mx().mx_fp4_quantize_act_slab(y)
    else:
        ref = mx().mx_quantize_act_slab(y)
    assert torch.equal(slab.q, ref.q) and torch.equal(slab.s, ref.s)
    assert R == (M + 255) // 256 * 256


@pytest.mark.parametrize("act", ["fp8", "fp4"])
@pytest.mark.parametrize("M", [9, 4101])
def test_in_place_strided_and_untouched_surroundings(M, act):
    print(f"norm in place M={M} {act}", flush=True)
    d = dev()
    K = 320
    g = torch.Generator(device=d).manual_seed(M)
    xb = torch.randn((M, K + 64), generator=g, device=d).to(torch.bfloat16)
    rb = torch.randn((M + 2, K + 32), generator=g, device=d)
    yb = torch.full((M + 2, K + 16), 9.0, dtype=torch.bfloat16, device=d)
    x, r, y = xb[:, 32 : 32 + K], rb[1 : M + 1, 16 : 16 + K], yb[1 : M + 1, 8 : 8 + K]
    r0, rb0 = r.clone(), rb.clone()
    plain, h0 = mx().mx_rmsnorm_slab(x.contiguous(), residual=r0, act=act)
    slab, h = mx().mx_rmsnorm_slab(x, residual=r, residual_out=r, act=act, y=y)
    assert h is r
    assert torch.equal(bits(r), bits(h0)) and torch.equal(slab.q, plain.q) and torch.equal(slab.s, plain.s)
    rb0[1 : M + 1, 16 : 16 + K] = h0
    assert torch.equal(bits(rb), bits(rb0))
    yy = yb.clone()
    yy[1 : M + 1, 8 : 8 + K] = 9.0
    assert bool((yy == 9.0).all())
    ref = (mx().mx_fp4_quantize_act_slab if act == "fp4" else mx().mx_quantize_act_slab)(y)
    assert torch.equal(ref.q, slab.q)


@pytest.mark.parametrize("M", [12, 4107])
def test_special_rows(M):
    print(f"norm special rows M={M}", flush=True)
    d = dev()
    K = 128
    x, _, w = inputs(M, K, None, torch.float32, 7)
    x[0] = 0
    x[1, 3] = float("nan")
    x[2, 70] = float("inf")
    x[3] = torch.finfo(torch.bfloat16).max  # squares far past f32
    x[4] = 2.0**-133  # squares far below f32
    x[5] = -0.0
    x[6, ::2] = -3.0e38
    for eps in (1e-6, 0.0):
        y = torch.empty((M, K), dtype=torch.bfloat16, device=d)
        slab, _ = mx().mx_rmsnorm_slab(x.to(d), w.to(d), eps=eps, y=y)
        n = 12
        _, ry = oracle.rmsnorm_ref(f64(x[:n]), None, f64(w), eps)
        assert np.array_equal(f64(y[:n]), ry, equal_nan=True), eps
        codes, scales = oracle.quantize_mx(ry)
        assert np.array_equal(u8(slab.s[:, :n]).transpose(1, 0, 2).reshape(n, -1), scales)
        assert np.array_equal(u8(slab.q[:, :n]).transpose(1, 0, 2).reshape(n, -1), codes)


def test_no_gain_dropped_outputs_and_empty():
    print("norm options", flush=True)
    d = dev()
    x, r, _ = inputs(33, 256, torch.bfloat16, None, 4)
    slab, h = mx().mx_rmsnorm_slab(x.to(d), residual=r.to(d))
    check(x, r, None, 1e-6, "fp8", slab, h, None, "no gain")
    # Through the C call: h not stored.
    m = mx()
    xd, rd = x.to(d), r.to(d)
    s2 = m.Slab(torch.empty_like(slab.q), torch.empty_like(slab.s), 33)
    m._run(m.lib().mx_rmsnorm_slab, xd.device, m._adr(xd), 256, m._adr(rd), 0, 256, m._adr(None), 0, 1e-6, 33, 256,
           m._adr(None), 0, m._adr(None), 0, 0, m._adr(s2.q), m._adr(s2.s))
    assert torch.equal(s2.q, slab.q) and torch.equal(s2.s, slab.s) and torch.equal(rd.cpu(), r)
    empty, h = m.mx_rmsnorm_slab(torch.empty((0, 64), dtype=torch.bfloat16, device=d))
    assert empty.q.numel() == 0 and h is None
