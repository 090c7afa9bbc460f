"""Plain float64 reference of the MXFP4 operators and of the RMS norm that
feeds a quantized linear.

TEST INFRASTRUCTURE ONLY: imported by ``tests/``, never by the product path,
and it imports nothing from the product package.

MXFP4 is the OCP microscaling format with E2M1 elements: one E8M0 scale per
32 elements along K, shared exponent floor(log2 amax) - 2 clamped to the E8M0
range, elements rounded to nearest with ties to the even code after saturation
to +-6, the sign of zero kept. A group holding NaN or Inf gets scale 0xFF and
every code 7. Every function is the definition written out with numpy.
"""

import numpy as np

from .mx_oracle import E8M0_BIAS, E8M0_NAN, GROUP, bf16_round, e8m0_decode, gelu_tanh

E2M1_EMAX = 2  # unbiased exponent of the top E2M1 binade
E2M1_MAGNITUDES = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e2m1_decode(codes):
    """Value of each E2M1 code (bit 3 the sign) as float64, sign of zero kept."""
    c = np.asarray(codes).astype(np.int64)
    mag = E2M1_MAGNITUDES[c & 7]
    return np.where(c & 8, -mag, mag)


def e2m1_encode(v):
    """E2M1 code of each float64 value: nearest magnitude, ties to the even
    code, saturating at 6; the sign bit is copied. NaN gives 7."""
    v = np.asarray(v, dtype=np.float64)
    a = np.minimum(np.abs(np.nan_to_num(v, nan=6.0, posinf=6.0, neginf=-6.0)), 6.0)
    d = np.abs(a[..., None] - E2M1_MAGNITUDES)  # exact: both have few bits near a tie
    best = d.min(axis=-1, keepdims=True)
    # The nearest magnitudes; of two at the same distance the even code.
    code = np.argmax(np.where(d == best, 2 - np.arange(8) % 2, 0), axis=-1)
    neg = np.signbit(v) & ~np.isnan(v)
    return (code | np.where(neg, 8, 0)).astype(np.uint8)


def fp4_scale_code(amax):
    """E8M0 code of the shared scale 2**(floor(log2 amax) - 2), clamped to
    [-127, 127]; 0xFF for a group that is not finite."""
    amax = np.asarray(amax, dtype=np.float64)
    _, p = np.frexp(np.nan_to_num(amax, nan=0.0, posinf=0.0))
    e = np.clip(np.where(amax > 0, p - 1 - E2M1_EMAX, -E8M0_BIAS), -127, 127)
    return np.where(np.isfinite(amax), e + E8M0_BIAS, E8M0_NAN).astype(np.uint8)


def quantize_fp4(x):
    """MXFP4 quantization along the last axis (a multiple of 32): codes uint8
    [..., K] (one per element) and scales uint8 [..., K/32]."""
    x = np.asarray(x, dtype=np.float64)
    K = x.shape[-1]
    if K % GROUP:
        raise ValueError("K must be a multiple of 32")
    g = x.reshape(x.shape[:-1] + (K // GROUP, GROUP))
    with np.errstate(invalid="ignore"):
        amax = np.max(np.abs(g), axis=-1)
    scales = fp4_scale_code(amax)
    codes = e2m1_encode(np.ldexp(g, -(scales.astype(np.int64) - E8M0_BIAS)[..., None]))
    codes[scales == E8M0_NAN] = 7
    return codes.reshape(x.shape), scales


def dequantize_fp4(codes, scales):
    """float64 value of MXFP4 data (NaN where the scale is)."""
    codes = np.asarray(codes)
    K = codes.shape[-1]
    vals = e2m1_decode(codes).reshape(codes.shape[:-1] + (K // GROUP, GROUP))
    return (vals * e8m0_decode(scales)[..., None]).reshape(codes.shape)


def pack_rows(codes):
    """Row-major packed codes [rows, K/2]: element 2b in the low half of byte b."""
    c = np.asarray(codes)
    return (c[..., 0::2] | (c[..., 1::2] << 4)).astype(np.uint8)


def fp4_slab(codes, scales):
    """The slab layout of [rows, K] codes and [rows, K/32] scales: uint8
    [S, R/16, 4, 16, 16] and [S, R, 4], R = rows rounded up to 256, S =
    ceil(K/128), everything past the operand zero."""
    rows, K = codes.shape
    R, S = (rows + 255) // 256 * 256, (K + 127) // 128
    q = np.zeros((S, R // 16, 4, 16, 16), dtype=np.uint8)
    s = np.zeros((S, R, 4), dtype=np.uint8)
    packed = pack_rows(codes)
    for g in range(K // GROUP):
        block = np.zeros((R, 16), dtype=np.uint8)
        block[:rows] = packed[:, 16 * g : 16 * g + 16]
        q[g // 4, :, g % 4] = block.reshape(R // 16, 16, 16)
        s[g // 4, :rows, g % 4] = scales[:, g]
    return q, s


def linear_values_ref(xh, wh, bias=None, epilogue="none"):
    """y* = phi(xh @ wh^T + bias) and S = |xh| @ |wh|^T in float64, on values."""
    y = xh @ wh.T
    S = np.abs(xh) @ np.abs(wh).T
    if bias is not None:
        y = y + np.asarray(bias, dtype=np.float64)[None, :]
    if epilogue == "gelu_tanh":
        y = gelu_tanh(y)
    elif epilogue != "none":
        raise ValueError(f"unknown epilogue {epilogue!r}")
    return y, S


def rmsnorm_ref(x, residual=None, gain=None, eps=1e-6, residual_f32=False):
    """(h, y): h = x + residual rounded to the residual's type (bf16, or
    float32), y = bf16(h * gain / sqrt(mean(h**2) + eps)), float64 arrays."""
    x = np.asarray(x, dtype=np.float64)
    with np.errstate(invalid="ignore", over="ignore", divide="ignore"):
        h = x
        if residual is not None:
            h = x + np.asarray(residual, dtype=np.float64)
            h = h.astype(np.float32).astype(np.float64) if residual_f32 else bf16_round(h)
        rstd = 1.0 / np.sqrt(np.mean(h * h, axis=-1, keepdims=True) + eps)
        y = h * rstd * (1.0 if gain is None else np.asarray(gain, dtype=np.float64))
        return h, bf16_round(y.astype(np.float32).astype(np.float64))
