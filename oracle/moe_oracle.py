"""Plain float64 references of the mixture-of-experts operators and of the norms
around a block.

TEST INFRASTRUCTURE ONLY: imported by ``tests/``, never by the product path,
and it imports nothing from the product package.

Every function is the definition in ``include/mx.h`` written out with numpy.
"""

import numpy as np

from .fp4_oracle import dequantize_fp4, e2m1_decode, e2m1_encode, fp4_scale_code, quantize_fp4
from .mx_oracle import E8M0_BIAS, GROUP, bf16_round, dequantize_mx, e4m3_decode, e4m3_encode, gelu_tanh, mx_scale_code
from .mx_oracle import quantize_mx

F32_MAX = float(np.finfo(np.float32).max)


def _f32(v):
    with np.errstate(over="ignore", invalid="ignore"):
        return np.asarray(v, dtype=np.float64).astype(np.float32).astype(np.float64)


def _best(keys, n):
    """Indices of the n highest keys, ties to the lower index."""
    return np.lexsort((np.arange(len(keys)), -keys))[:n]


def route_ref(logits, k, scores="softmax", bias=None, groups=1, top_groups=1, renorm=True, scale=1.0):
    """(ids int64 [T, k], weights float64 [T, k]) of mx_route, token by token."""
    L = np.asarray(logits, dtype=np.float64)
    T, E = L.shape
    ids, weights = np.empty((T, k), np.int64), np.empty((T, k))
    for t in range(T):
        row = np.where(np.isnan(L[t]), -np.inf, np.minimum(L[t], F32_MAX))
        live = row > -np.inf
        s = np.zeros(E)
        with np.errstate(over="ignore", invalid="ignore"):
            if scores == "sigmoid":
                s[live] = 1.0 / (1.0 + np.exp(-row[live]))
            elif live.any():
                p = np.exp(row[live] - row[live].max())
                s[live] = p / p.sum()
            c = row if bias is None else np.where(live, _f32(s + np.asarray(bias, dtype=np.float64)), -np.inf)
        c = np.where(np.isnan(c), -np.inf, c)
        if groups > 1:
            g = -np.sort(-c.reshape(groups, -1), axis=1)
            gs = g[:, 0].copy()
            if bias is not None and g.shape[1] > 1:
                with np.errstate(over="ignore", invalid="ignore"):
                    gs = np.where(g[:, 1] > -np.inf, _f32(g[:, 0] + np.where(g[:, 1] > -np.inf, g[:, 1], 0.0)), gs)
            gs = np.where(np.isnan(gs), -np.inf, gs)
            kept = np.zeros(groups, bool)
            kept[_best(gs, top_groups)] = True
            c = np.where(np.repeat(kept, E // groups), c, -np.inf)
        ids[t] = _best(c, k)
        w = np.where(c[ids[t]] > -np.inf, s[ids[t]], 0.0)
        if renorm:
            w = w / w.sum() if w.sum() > 0 else np.zeros(k)
        weights[t] = w * scale
    return ids, weights


def silu(x):
    with np.errstate(over="ignore"):
        return x / (1.0 + np.exp(-x))


# Largest slopes of the gates, each rounded up.
GATES = {"silu": (silu, 1.1), "gelu": (gelu_tanh, 1.13)}


def _codec(act):
    if act == "fp4":
        return quantize_fp4, dequantize_fp4, fp4_scale_code, e2m1_encode, e2m1_decode
    return quantize_mx, dequantize_mx, mx_scale_code, e4m3_encode, e4m3_decode


def activation_values(x, act):
    """Values of the MX quantization of x."""
    q, d = _codec(act)[:2]
    return d(*q(x))


def _quantized_range(lo, hi, act):
    """Per element the lowest and highest value that the quantization of bf16 rows
    between lo and hi (bf16 values, lo <= hi) can take."""
    _, _, scale_code, encode, decode = _codec(act)
    shp = lo.shape[:-1] + (lo.shape[-1] // GROUP, GROUP)
    a = np.maximum(np.abs(lo), np.abs(hi)).reshape(shp)
    b = np.where((lo <= 0) & (hi >= 0), 0.0, np.minimum(np.abs(lo), np.abs(hi))).reshape(shp)
    shi = scale_code(a.max(axis=-1)).astype(np.int64)
    slo = scale_code(b.max(axis=-1)).astype(np.int64)
    qlo, qhi = np.full(shp, np.inf), np.full(shp, -np.inf)
    for d in range(int((shi - slo).max()) + 1):
        step = np.ldexp(1.0, np.minimum(slo + d, shi)[..., None] - E8M0_BIAS)
        qlo = np.minimum(qlo, decode(encode(lo.reshape(shp) / step)) * step)
        qhi = np.maximum(qhi, decode(encode(hi.reshape(shp) / step)) * step)
    return qlo.reshape(lo.shape), qhi.reshape(lo.shape)


def experts_ref(x, ids, weights, up, down, act, gate):
    """(y*, tol) of mx_fp4_experts on values: x float64 [T, H] (bf16 values), up
    [E, 2 I, H] and down [E, H, I] the weights' values.

    tol bounds the library's error, bf16 rounding included:
      - a product's fp32 sum is within r S of the exact one, S the sum of its terms'
        magnitudes: r = 2^-14 for exact products (at most K/64 + 64 roundings of
        2^-24; 2^-15.7 at K = 16384), 2^-12 more with MXFP8 activations, whose
        products the matrix cores cut (include/mx.h);
      - a = gate(g) u then moves by |gate'| r S_g |u| + |gate| r S_u + both errors'
        product, and by 2^-20 of itself in its own evaluation;
      - h may round to any value between the quantizations of the ends of that range;
      - o moves by those steps times |down|, by r S_o, and by its f16 form: half a step
        of 2^-11, and 2^-38 of the largest of 32 columns where it is that much smaller;
      - the weighted sum adds k + 1 roundings of 2^-24; half a bf16 step at the end."""
    f, slope = GATES[gate]
    r = 2.0**-14 + (2.0**-12 if act == "fp8" else 0.0)
    T, H = x.shape
    E, _, I = down.shape
    xh = activation_values(x, act)
    y, tol, mag = np.zeros((T, H)), np.zeros((T, H)), np.zeros((T, H))
    for e in range(E):
        rows, slots = np.nonzero(ids == e)
        if rows.size == 0:
            continue
        v = xh[rows]
        u, S = v @ up[e].T, np.abs(v) @ np.abs(up[e]).T
        g, u, rg, ru = u[:, :I], u[:, I:], r * S[:, :I], r * S[:, I:]
        a = f(g) * u
        ra = slope * rg * np.abs(u) + np.abs(f(g)) * ru + slope * rg * ru + 2.0**-20 * np.abs(a)
        h = activation_values(bf16_round(a), act)
        lo, hi = _quantized_range(bf16_round(a - ra), bf16_round(a + ra), act)
        delta = np.maximum(hi - h, h - lo)
        o, So = h @ down[e].T, (np.abs(h) + delta) @ np.abs(down[e]).T
        ro = delta @ np.abs(down[e]).T + r * So
        top = np.repeat((np.abs(o) + ro).reshape(len(rows), -1, GROUP).max(axis=-1), GROUP, axis=-1)
        ro += 2.0**-11 * (np.abs(o) + ro) + 2.0**-38 * top
        w = weights[rows, slots][:, None]
        np.add.at(y, rows, w * o)
        np.add.at(tol, rows, np.abs(w) * ro)
        np.add.at(mag, rows, np.abs(w) * (np.abs(o) + ro))
    tol += (ids.shape[1] + 1) * 2.0**-24 * mag
    return y, tol + 2.0**-8 * (np.abs(y) + tol) + 2.0**-134


def block_h_ref(x, residual, residual_scale=1.0, post=False, post_weight=None, gate=None, eps=1e-6):
    """(h before its rounding, the sum of its terms' magnitudes), float64; gate rows
    already one a row of x, or [1, K]."""
    n = np.asarray(x, dtype=np.float64)
    with np.errstate(invalid="ignore", divide="ignore"):
        if post:
            n = n / np.sqrt(np.mean(n * n, axis=-1, keepdims=True) + eps)
            if post_weight is not None:
                n = n * post_weight
        if gate is not None:
            n = n * gate
        r = np.float64(residual_scale) * np.asarray(residual, dtype=np.float64)
        return r + n, np.abs(r) + np.abs(n)


def block_y_ref(h, kind="rms", weight=None, scale=None, shift=None, eps=1e-6):
    """(y before its rounding, a bound that f32 arithmetic before it would keep) from h
    as stored, float64.

    The library computes in float64, so its own error is far smaller
    (tests/test_gpu_block_norm_exact.py derives that bound). The one here counts f32
    roundings of 2^-24 of a term: a row's sum of squares 8 (its f32 sums of 8; their sum
    is f64) and its differences from the mean 4, halved by the root, rstd 1, products
    and the shift 6: under 2^-19 of the difference's term. A mean is off by 8 2^-24 of
    the mean magnitude, in the difference and (again) in the squares: under 2^-20 of it."""
    h = np.asarray(h, dtype=np.float64)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        m = np.mean(h, axis=-1, keepdims=True) if kind == "layer" else 0.0
        d = h - m
        rstd = 1.0 / np.sqrt(np.mean(d * d, axis=-1, keepdims=True) + eps)
        factor = rstd * (1.0 if weight is None else weight) * (1.0 if scale is None else 1.0 + scale)
        y = d * factor
        err = np.abs(factor) * np.abs(d) * 2.0**-19
        if scale is not None:  # 1 + scale may cancel: its two terms are rounded apart
            err = err + np.abs(d * rstd * (1.0 if weight is None else weight)) * (1.0 + np.abs(scale)) * 2.0**-22
        if kind == "layer":
            mean_abs = np.mean(np.abs(h), axis=-1, keepdims=True)
            err = err + np.abs(factor) * mean_abs * 2.0**-20
        if shift is not None:
            y = y + shift
            err = err + (np.abs(y) + np.abs(shift)) * 2.0**-23
        return y, err
