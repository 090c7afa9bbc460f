"""Measured operators: 4-bit microscaled (MXFP4) linears, their quantizer, and
the residual RMS norm that feeds a quantized linear.

Formats (both with one E8M0 scale 2**e per 32 elements along K):
  MXFP8  E4M3 elements, e = clamp(floor(log2 amax) - 8, -127, 127)
  MXFP4  E2M1 elements, e = clamp(floor(log2 amax) - 2, -127, 127)
  element = nearest representable x * 2**-e after saturation, ties to even.

Slab layouts, R = rows rounded up to 256, rows past the last are zero:
  MXFP8  codes uint8 [K/64, R, 64], scales uint8 [K/64, R, 2]
  MXFP4  codes uint8 [ceil(K/128), R/16, 4, 16, 16]: slab, block of 16 rows,
         group of 32 elements, row, byte (element 2b of the group in the low
         half of byte b, 2b + 1 in the high half); scales uint8
         [ceil(K/128), R, 4]; groups past K are zero

`own = False` computes each operator in elementary torch operations; `own =
True` makes the library's calls on the same data.
"""

import math

import torch

own = False

DEV = "cuda"
GROUP = 32
# The shapes of the Wan2.2-A14B transformer that the repository's linears
# come from: hidden size, FFN size, video tokens, text tokens.
HIDDEN, FFN, VIDEO, TEXT = 5120, 13824, 75348, 512
EPS = 1e-6


def listed():
    return [
        # Residual add, RMS norm and MXFP8 codes ahead of a quantized linear.
        {"name": "norm8_decode", "op": "norm8", "M": 1, "K": HIDDEN, "res": "bf16"},  # one decoded token
        {"name": "norm8_text", "op": "norm8", "M": 509, "K": 4096, "res": "f32"},  # a prompt, fp32 residual stream
        {"name": "norm8_video", "op": "norm8", "M": VIDEO, "K": HIDDEN, "res": "bf16"},  # every video token
        # MXFP4 quantization followed by dequantization: what a calibration
        # pass over weights (fp32) or activations (bf16) runs.
        {"name": "quant4_act", "op": "quant4", "M": 333, "K": HIDDEN, "src": "bf16"},
        {"name": "quant4_weight", "op": "quant4", "M": FFN, "K": HIDDEN, "src": "f32"},
        # MXFP4 weights, MXFP4 activations quantized at run time.
        {"name": "w4a4_decode", "op": "linear", "act": "fp4", "M": 1, "K": HIDDEN, "N": HIDDEN, "gelu": False},
        {"name": "w4a4_text", "op": "linear", "act": "fp4", "M": TEXT, "K": HIDDEN, "N": 2 * HIDDEN, "gelu": False},
        {"name": "w4a4_video_qkv", "op": "linear", "act": "fp4", "M": VIDEO, "K": HIDDEN, "N": 3 * HIDDEN, "gelu": False},
        # MXFP4 weights, MXFP8 activations: small batches being decoded, then
        # a prompt.
        {"name": "w4a8_decode_ffn", "op": "linear", "act": "fp8", "M": 7, "K": HIDDEN, "N": FFN, "gelu": True},
        {"name": "w4a8_batch", "op": "linear", "act": "fp8", "M": 128, "K": FFN, "N": HIDDEN, "gelu": False},
        {"name": "w4a8_prompt", "op": "linear", "act": "fp8", "M": 4001, "K": HIDDEN, "N": HIDDEN, "gelu": False},
        # The norm writing MXFP4 codes, and the projection that reads them.
        {"name": "norm4_proj", "op": "norm4_linear", "M": 300, "K": HIDDEN, "N": 3 * HIDDEN, "res": "bf16"},
    ]


def _logint(rng, lo, hi, step):
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(step, int(round(v / step)) * step)


def draw(rng):
    op = rng.choice(["norm8", "quant4", "w4a4", "w4a8", "w4a4", "w4a8", "norm4_linear"])
    if op == "norm8":
        return {"op": "norm8", "M": _logint(rng, 1, 40000, 1), "K": _logint(rng, 512, 16384, 64),
                "res": rng.choice(["bf16", "f32", "none"])}
    if op == "quant4":
        return {"op": "quant4", "M": _logint(rng, 1, 20000, 1), "K": _logint(rng, 512, 16384, 32),
                "src": rng.choice(["bf16", "f32"])}
    if op == "norm4_linear":
        return {"op": op, "M": _logint(rng, 1, 4000, 1), "K": _logint(rng, 1024, 8192, 32),
                "N": _logint(rng, 1024, 16384, 16), "res": rng.choice(["bf16", "f32", "none"])}
    return {"op": "linear", "act": "fp4" if op == "w4a4" else "fp8", "M": _logint(rng, 1, 24000, 1),
            "K": _logint(rng, 1024, 14336, 32 if op == "w4a4" else 64), "N": _logint(rng, 1024, 16384, 16),
            "gelu": rng.random() < 0.3}


def work(case):
    M, K = case["M"], case["K"]
    res = {"bf16": 4 * M * K, "f32": 8 * M * K, "none": 0}[case.get("res", "none")]  # residual read and written
    if case["op"] == "norm8":
        return {"bytes": 2 * M * K + res + 2 * K + M * K + M * K // 32, "flops": 4 * M * K}
    if case["op"] == "quant4":
        return {"bytes": (4 if case["src"] == "f32" else 2) * M * K + 2 * M * K, "flops": 4 * M * K}
    N = case["N"]
    weights = N * K // 2 + N * K // 32 + 2 * N
    extra = res + 2 * K if case["op"] == "norm4_linear" else 0
    return {"bytes": 2 * M * K + weights + 2 * M * N + extra, "flops": 2 * M * N * K}


# ---------------------------------------------------------------------------
# Inputs.


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _activation(M, K, g):
    """N(0, 1) with one entry in a thousand 50 times larger, as activations have."""
    x = torch.randn((M, K), generator=g, device=DEV)
    out = torch.rand((M, K), generator=g, device=DEV) < 1e-3
    return torch.where(out, 50.0 * x, x).to(torch.bfloat16)


def prepare(case, seed):
    g = _gen(seed)
    M, K, op = case["M"], case["K"], case["op"]
    st = {"case": dict(case)}
    if op == "quant4":
        if case["src"] == "f32":
            st["x"] = 0.02 * torch.randn((M, K), generator=g, device=DEV)
        else:
            st["x"] = _activation(M, K, g)
        return st
    st["x"] = _activation(M, K, g)
    if op in ("norm8", "norm4_linear"):
        st["gain"] = (1.0 + 0.1 * torch.randn((K,), generator=g, device=DEV)).to(torch.bfloat16)
        res = case["res"]
        st["residual"] = None
        if res != "none":
            r = 3.0 * torch.randn((M, K), generator=g, device=DEV)
            st["residual"] = r.to(torch.bfloat16) if res == "bf16" else r
    if op in ("linear", "norm4_linear"):
        N = case["N"]
        # The weights a program keeps: MXFP4 codes and scales in slabs.
        v, e = _quantize(0.02 * torch.randn((N, K), generator=g, device=DEV), "fp4")
        st["wq"], st["ws"] = _pack4(v, e)
        st["bias"] = (0.01 * torch.randn((N,), generator=g, device=DEV)).to(torch.float16)
    return st


# ---------------------------------------------------------------------------
# Plain form.


def _pow2(e):
    """2**e as float32 for integer e in [-126, 127]."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _quantize(x, fmt):
    """Microscaled quantization of float32 [rows, K]: element values before
    the scale [rows, K/32, 32] and exponents e [rows, K/32]."""
    g = x.view(x.shape[0], -1, GROUP)
    amax = g.abs().amax(dim=-1)
    p = torch.frexp(amax).exponent.to(torch.int32) - 1
    e = torch.where(amax > 0, p - (2 if fmt == "fp4" else 8), torch.full_like(p, -127)).clamp(-127, 127)
    v = g * _pow2(-e)[..., None]
    if fmt == "fp8":
        return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).to(torch.float32), e
    a = v.abs()
    # E2M1 magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6: steps of 0.5, 1 and 2.
    r = torch.where(a < 2, torch.round(a * 2) / 2, torch.where(a < 4, torch.round(a), torch.round(a / 2) * 2))
    return torch.copysign(r.clamp(max=6.0), v), e


def _scaled(v, e):
    """Values of quantized data, float32 [rows, K]."""
    s = torch.where(e > -127, _pow2(e.clamp(min=-126)), torch.full_like(v[..., 0], 2.0**-127))
    return (v * s[..., None]).view(v.shape[0], -1)


def _rows(n):
    return (n + 255) // 256 * 256


def _pack4(v, e):
    rows, groups = e.shape
    S, R = (groups + 3) // 4, _rows(rows)
    a = v.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code |= torch.signbit(v).to(torch.uint8) << 3
    byte = (code[..., 0::2] | (code[..., 1::2] << 4)).view(rows, groups * 16)
    q = torch.zeros((R, S * 64), dtype=torch.uint8, device=v.device)
    q[:rows, : groups * 16] = byte
    q = q.view(R // 16, 16, S, 4, 16).permute(2, 0, 3, 1, 4).contiguous()
    s = torch.zeros((R, S * 4), dtype=torch.uint8, device=v.device)
    s[:rows, :groups] = (e + 127).to(torch.uint8)
    return q, s.view(R, S, 4).transpose(0, 1).contiguous()


def _unpack4(q, s, rows, K):
    """Values of an MXFP4 slab, float32 [rows, K]."""
    b = q.permute(1, 3, 0, 2, 4).reshape(q.shape[1] * 16, -1)[:rows, : K // 2]
    code = torch.stack((b & 15, b >> 4), dim=-1).view(rows, K)
    m = (code & 7).to(torch.float32)
    a = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
    v = torch.where(code >= 8, -a, a).view(rows, K // GROUP, GROUP)
    e = s[:, :rows].transpose(0, 1).reshape(rows, -1)[:, : K // GROUP].to(torch.int32) - 127
    return _scaled(v, e)


def _pack8(v, e):
    rows, groups = e.shape
    S, R = groups // 2, _rows(rows)
    q = torch.zeros((S, R, 64), dtype=torch.uint8, device=v.device)
    q[:, :rows] = v.to(torch.float8_e4m3fn).view(torch.uint8).view(rows, S, 64).transpose(0, 1)
    s = torch.zeros((S, R, 2), dtype=torch.uint8, device=v.device)
    s[:, :rows] = (e + 127).to(torch.uint8).view(rows, S, 2).transpose(0, 1)
    return q, s


def _norm(x, residual, gain):
    """(new residual or None, bf16 RMS norm of it); the mean square and the
    product in 64 bits, since the result is next rounded to few bits."""
    if residual is not None:
        h = (x.to(torch.float32) + residual.to(torch.float32)).to(residual.dtype)
    else:
        h = x
    d = h.to(torch.float64)
    y = d * (1.0 / torch.sqrt((d * d).mean(dim=-1, keepdim=True) + EPS)) * gain.to(torch.float64)
    return (h if residual is not None else None), y.to(torch.float32).to(torch.bfloat16)


def _product(xv, wv, bias, gelu):
    y = torch.mm(xv, wv.t()) + bias.to(torch.float32)
    if gelu:
        y = 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))
    return y.to(torch.bfloat16)


def _plain(st):
    c, x = st["case"], st["x"]
    if c["op"] == "quant4":
        return _scaled(*_quantize(x.to(torch.float32), "fp4")).to(torch.bfloat16)
    if c["op"] == "norm8":
        h, y = _norm(x, st["residual"], st["gain"])
        q, s = _pack8(*_quantize(y.to(torch.float32), "fp8"))
        return {"residual": h, "codes": q.view(torch.float8_e4m3fn), "scales": s.view(torch.float8_e8m0fnu)}
    wv = _unpack4(st["wq"], st["ws"], c["N"], c["K"])
    if c["op"] == "linear":
        xv = _scaled(*_quantize(x.to(torch.float32), c["act"]))
        return _product(xv, wv, st["bias"], c["gelu"])
    h, y = _norm(x, st["residual"], st["gain"])
    xv = _scaled(*_quantize(y.to(torch.float32), "fp4"))
    return {"residual": h, "y": _product(xv, wv, st["bias"], False)}


# ---------------------------------------------------------------------------
# The library's calls.


def _library(st):
    import mxfp8_w8a8_quantized_amd as mx

    c, x = st["case"], st["x"]
    if c["op"] == "quant4":
        quantize = mx.mx_fp4_quantize_weight_slab if c["src"] == "f32" else mx.mx_fp4_quantize_act_slab
        return mx.mx_fp4_dequantize_slab(quantize(x))
    if c["op"] == "norm8":
        slab, h = mx.mx_rmsnorm_slab(x, st["gain"], residual=st["residual"], eps=EPS)
        return {"residual": h, "codes": slab.q.view(torch.float8_e4m3fn), "scales": slab.s.view(torch.float8_e8m0fnu)}
    w = mx.FP4Slab(st["wq"], st["ws"], c["N"], c["K"])
    if c["op"] == "linear":
        return mx.mx_fp4_linear(x, w, st["bias"], gelu=c["gelu"], act=c["act"])
    slab, h = mx.mx_rmsnorm_slab(x, st["gain"], residual=st["residual"], eps=EPS, act="fp4")
    return {"residual": h, "y": mx.mx_fp4_linear_slab(slab, w, st["bias"])}


def run(state):
    return _library(state) if own else _plain(state)


# ---------------------------------------------------------------------------
# The definition in 64 bits, from the representable values themselves.

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _exact_exponent(g, top):
    amax = g.abs().amax(dim=-1)
    # The exponent field of a float64 is floor(log2) + 1023.
    field = ((amax.view(torch.int64) >> 52) & 0x7FF) - 1023
    return torch.where(amax > 0, field - top, torch.full_like(field, -127)).clamp(-127, 127)


def _exact_pow2(e):
    return ((e + 1023) << 52).view(torch.float64)


def _exact_values(x, fmt):
    """float64 [rows, K] -> values of its microscaled quantization, float64."""
    g = x.view(x.shape[0], -1, GROUP)
    e = _exact_exponent(g, 2 if fmt == "fp4" else 8)
    v = g * _exact_pow2(-e)[..., None]
    a = v.abs()
    if fmt == "fp4":
        # Each midpoint between neighbours is crossed upwards strictly, or at
        # the midpoint itself where the upper neighbour has the even code.
        q = torch.zeros_like(a)
        for i in range(7):
            mid, step = 0.5 * (_E2M1[i] + _E2M1[i + 1]), _E2M1[i + 1] - _E2M1[i]
            q += step * ((a >= mid) if (i + 1) % 2 == 0 else (a > mid)).to(torch.float64)
    else:
        ex = (((a.view(torch.int64) >> 52) & 0x7FF) - 1023).clamp(min=-6)
        step = _exact_pow2(ex - 3)
        q = (torch.round(a / step) * step).clamp(max=448.0)
    return torch.copysign(q, v), e


def _exact_quantized(x, fmt):
    q, e = _exact_values(x, fmt)
    return (q * _exact_pow2(e)[..., None]).view(x.shape)


def _exact_weights(st, N, K):
    table = torch.tensor(_E2M1 + tuple(-v for v in _E2M1), dtype=torch.float64, device=DEV)
    out = torch.empty((N, K), dtype=torch.float64, device=DEV)
    q, s = st["wq"], st["ws"]
    for k0 in range(0, K, 128):
        n = min(128, K - k0)
        b = torch.cat([q[k0 // 128, :, c].reshape(-1, 16) for c in range(n // 32)], dim=1)[:N].to(torch.int64)
        sc = _exact_pow2(s[k0 // 128, :N, : n // 32].to(torch.int64) - 127).repeat_interleave(GROUP, dim=1)
        out[:, k0 : k0 + n : 2] = table[b & 15]
        out[:, k0 + 1 : k0 + n : 2] = table[b >> 4]
        out[:, k0 : k0 + n] *= sc
    return out


def _exact_norm(st):
    x, r = st["x"].to(torch.float64), st["residual"]
    h = x if r is None else (x + r.to(torch.float64)).to(r.dtype)
    d = h.to(torch.float64)
    rms = torch.sqrt(torch.sum(d * d, dim=1) / d.shape[1] + EPS)
    y = (d / rms[:, None] * st["gain"].to(torch.float64)[None, :]).to(torch.float32).to(torch.bfloat16)
    return (None if r is None else d), y.to(torch.float64)


def exact(case, seed):
    st = prepare(case, seed)
    M, K, op = case["M"], case["K"], case["op"]
    if op == "quant4":
        return _exact_quantized(st["x"].to(torch.float64), "fp4")
    if op == "norm8":
        h, y = _exact_norm(st)
        q, e = _exact_values(y, "fp8")
        R = _rows(M)
        codes = torch.zeros((K // 64, R, 64), dtype=torch.float64, device=DEV)
        codes[:, :M] = q.view(M, K // 64, 64).transpose(0, 1)
        scales = torch.full((K // 64, R, 2), 2.0**-127, dtype=torch.float64, device=DEV)
        scales[:, :M] = _exact_pow2(e).view(M, K // 64, 2).transpose(0, 1)
        return {"residual": h, "codes": codes, "scales": scales}
    h = None
    if op == "linear":
        xv = _exact_quantized(st["x"].to(torch.float64), case["act"])
    else:
        h, y = _exact_norm(st)
        xv = _exact_quantized(y, "fp4")
    out = torch.mm(xv, _exact_weights(st, case["N"], K).t())
    out += st["bias"].to(torch.float64)
    if case.get("gelu"):
        out = 0.5 * out * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (out + 0.044715 * out**3)))
    return out if op == "linear" else {"residual": h, "y": out}
