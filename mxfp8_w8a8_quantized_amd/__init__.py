"""MXFP8 W8A8 linear layer for AMD Instinct MI355X (gfx950).

Thin Python binding of the C ABI in ``include/mx.h`` (same names). It only
marshals arguments: torch tensors in, device pointers and the current HIP
stream out; every step of the computation runs in the library's HIP kernels.
If the built library ``libmxfp8.so`` is missing, every call raises.
"""

import ctypes
import functools
import os
from typing import NamedTuple

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "libmxfp8.so")

MX_ABI_VERSION = 12
MX_OK = 0
MX_ERR_INVALID_ARGUMENT = 1
MX_ERR_UNSUPPORTED = 2
MX_ERR_HIP = 3
MX_EPI_NONE = 0
MX_EPI_GELU_TANH = 1
MX_DT_BF16 = 0
MX_DT_F32 = 1
MX_ACT_FP8 = 0
MX_ACT_FP4 = 1
ACT_FORMATS = {"fp8": MX_ACT_FP8, "fp4": MX_ACT_FP4}
MX_PLAN_SLAB = 0
MX_PLAN_SPLITK = 1
MX_PLAN_SMALL = 2
MX_PLAN_BALANCED = 3
MX_PLAN_SLAB_M128 = 4
PLAN_NAMES = {MX_PLAN_SLAB: "slab", MX_PLAN_SPLITK: "splitk", MX_PLAN_SMALL: "small", MX_PLAN_BALANCED: "balanced",
              MX_PLAN_SLAB_M128: "slab_m128"}
PLAN_KINDS = {v: k for k, v in PLAN_NAMES.items()}

# Every symbol include/mx.h declares, with its ctypes signature.
_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_INT = ctypes.c_int
_PI = ctypes.POINTER(ctypes.c_int)
SIGNATURES = {
    "mx_abi_version": ([], _INT),
    "mx_status_string": ([_INT], ctypes.c_char_p),
    "mx_last_hip_error": ([], _INT),
    "mx_last_error_message": ([], ctypes.c_char_p),
    "mx_quantize_act": ([_P, _I64, _I64, _I64, _P, _P, _P], _INT),
    "mx_quantize_weight": ([_P, _INT, _I64, _I64, _I64, _P, _P, _P], _INT),
    "mx_linear_fused": ([_P, _I64, _I64, _P, _P, _I64, _P, _INT, _P, _P], _INT),
    "mx_linear_q": ([_P, _P, _I64, _I64, _P, _P, _I64, _P, _INT, _P, _P], _INT),
    "mx_slab_rows": ([_I64], _I64),
    "mx_quantize_act_slab": ([_P, _I64, _I64, _I64, _P, _P, _P], _INT),
    "mx_quantize_weight_slab": ([_P, _INT, _I64, _I64, _I64, _P, _P, _P], _INT),
    "mx_slab_pack": ([_P, _P, _I64, _I64, _P, _P, _P], _INT),
    "mx_linear_slab": ([_P, _P, _I64, _I64, _P, _P, _I64, _P, _INT, _P, _P], _INT),
    "mx_linear_slab_m128": ([_P, _P, _I64, _I64, _P, _P, _I64, _P, _INT, _P, _P], _INT),
    "mx_linear_slab_requant": ([_P, _P, _I64, _I64, _P, _P, _I64, _P, _INT, _P, _P, _P], _INT),
    "mx_linear_splitk_ws_bytes": ([_I64, _I64, _INT], _I64),
    "mx_linear_splitk_choose": ([_I64, _I64, _I64], _INT),
    "mx_linear_slab_splitk": ([_P, _P, _I64, _I64, _P, _P, _I64, _P, _INT, _P, _INT, _P, _I64, _P], _INT),
    "mx_linear_small_ws_bytes": ([_I64, _I64, _INT], _I64),
    "mx_linear_small_choose": ([_I64, _I64, _I64], _INT),
    "mx_linear_slab_small": ([_P, _P, _I64, _I64, _P, _P, _I64, _P, _INT, _P, _INT, _P, _I64, _P], _INT),
    "mx_linear_balanced_ws_bytes": ([_I64, _I64, _I64], _I64),
    "mx_linear_slab_balanced": ([_P, _P, _I64, _I64, _P, _P, _I64, _P, _INT, _P, _P, _I64, _P], _INT),
    "mx_linear_plan_default": ([_I64, _I64, _I64, _PI, _PI], _INT),
    "mx_linear_plan_ws_bytes": ([_INT, _INT, _I64, _I64, _I64], _I64),
    "mx_linear_slab_plan": ([_INT, _INT, _P, _P, _I64, _I64, _P, _P, _I64, _P, _INT, _P, _P, _I64, _P], _INT),
    "mx_linear_tune_ws_bytes": ([_I64, _I64, _I64], _I64),
    "mx_linear_tune": ([_P, _P, _I64, _I64, _P, _P, _I64, _P, _INT, _P, _P, _I64, _INT, _P, _PI, _PI], _INT),
    "mx_linear_plan_lookup": ([_I64, _I64, _I64, _INT, _PI, _PI], _INT),
    "mx_linear_slab_auto": ([_P, _P, _I64, _I64, _P, _P, _I64, _P, _INT, _P, _P, _I64, _P], _INT),
    "mx_linear_plan_clear": ([], None),
    "mx_linear_ws_bytes": ([_I64, _I64, _I64], _I64),
    "mx_linear": ([_P, _I64, _I64, _I64, _P, _P, _I64, _P, _INT, _P, _P, _I64, _P], _INT),
    "mx_linear_noalloc": ([_P, _I64, _I64, _I64, _P, _P, _I64, _P, _INT, _P, _P], _INT),
    "mx_probe_mfma": ([_P, _P, _I64, _INT, _INT, _P, _P], _INT),
    "mx_pc_quantize_act_slab": ([_P, _I64, _I64, _I64, _P, _P, _P], _INT),
    "mx_pc_quantize_weight_slab": ([_P, _INT, _I64, _I64, _I64, _P, _P, _P], _INT),
    "mx_pc_linear_slab": ([_P, _P, _I64, _I64, _P, _P, _I64, _P, _INT, _P, _P], _INT),
    "mx_fp4_quantize_act_slab": ([_P, _I64, _I64, _I64, _P, _P, _P], _INT),
    "mx_fp4_quantize_weight_slab": ([_P, _INT, _I64, _I64, _I64, _P, _P, _P], _INT),
    "mx_fp4_dequantize_slab": ([_P, _P, _I64, _I64, _P, _INT, _I64, _P], _INT),
    "mx_fp4_slab_pack": ([_P, _P, _I64, _I64, _P, _P, _P], _INT),
    "mx_fp4_slab_unpack": ([_P, _P, _I64, _I64, _P, _P, _P], _INT),
    "mx_fp4_linear_slab": ([_INT, _P, _P, _I64, _I64, _P, _P, _I64, _P, _INT, _P, _P], _INT),
    "mx_fp4_linear_ws_bytes": ([_I64, _I64, _I64, _INT], _I64),
    "mx_fp4_linear_tile": ([_I64, _I64, _I64, _INT, _PI, _PI, _PI], _INT),
    "mx_fp4_linear": ([_P, _I64, _I64, _I64, _P, _P, _I64, _P, _INT, _INT, _P, _P, _I64, _P], _INT),
    "mx_rmsnorm_slab": ([_P, _I64, _P, _INT, _I64, _P, _INT, ctypes.c_double, _I64, _I64, _P, _I64, _P, _I64, _INT, _P,
                         _P, _P], _INT),
}


class MXError(RuntimeError):
    def __init__(self, status, message):
        self.status = status
        super().__init__(message)


_lib = None


def lib():
    """The loaded library (raises if it has not been built, or if it was built
    from other sources: another ABI version, or a call missing)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise MXError(-1, f"{LIB_PATH} is not built; run __graft_entry__.build()")
        handle = ctypes.CDLL(LIB_PATH)
        missing = [name for name in SIGNATURES if not hasattr(handle, name)]
        if missing:
            raise MXError(-1, f"{LIB_PATH} is out of date (no {missing[0]}); run __graft_entry__.build()")
        if handle.mx_abi_version() != MX_ABI_VERSION:
            raise MXError(-1, f"{LIB_PATH} is out of date (ABI version {handle.mx_abi_version()}, not "
                              f"{MX_ABI_VERSION}); run __graft_entry__.build()")
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(handle, name)
            fn.argtypes = args
            fn.restype = res
        _lib = handle
    return _lib


def _check(status):
    if status != MX_OK:
        L = lib()
        msg = L.mx_last_error_message().decode()
        name = L.mx_status_string(status).decode()
        raise MXError(status, f"{name}: {msg}")


def _ptr(t):
    return ctypes.c_void_p(t.data_ptr()) if t is not None and t.numel() > 0 else ctypes.c_void_p(0)


def _stream(device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need(t, name, dtype, device):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def mx_abi_version():
    return lib().mx_abi_version()


def mx_status_string(status):
    return lib().mx_status_string(status).decode()


def mx_last_hip_error():
    return lib().mx_last_hip_error()


def mx_last_error_message():
    return lib().mx_last_error_message().decode()


def mx_quantize_act(x, q=None, s=None):
    """bf16 [M, K] (rows may be strided) -> (codes uint8 [M, K], scales uint8 [M, K/32])."""
    if x.dim() != 2 or x.dtype != torch.bfloat16 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D bf16 tensor with unit column stride")
    M, K = x.shape
    dev = x.device
    q = torch.empty((M, K), dtype=torch.uint8, device=dev) if q is None else q
    s = torch.empty((M, K // 32), dtype=torch.uint8, device=dev) if s is None else s
    _need(q, "q", torch.uint8, dev)
    _need(s, "s", torch.uint8, dev)
    ld = x.stride(0) if M > 1 else K
    with torch.cuda.device(dev):
        _check(lib().mx_quantize_act(_ptr(x), M, K, ld, _ptr(q), _ptr(s), _stream(dev)))
    return q, s


def mx_quantize_weight(w, q=None, s=None):
    """fp32 or bf16 [N, K] -> (codes uint8 [N, K], scales uint8 [N, K/32])."""
    if w.dim() != 2 or w.stride(1) != 1:
        raise ValueError("w must be 2-D with unit column stride")
    dt = {torch.float32: MX_DT_F32, torch.bfloat16: MX_DT_BF16}.get(w.dtype)
    if dt is None:
        raise TypeError(f"w must be float32 or bfloat16, got {w.dtype}")
    N, K = w.shape
    dev = w.device
    q = torch.empty((N, K), dtype=torch.uint8, device=dev) if q is None else q
    s = torch.empty((N, K // 32), dtype=torch.uint8, device=dev) if s is None else s
    _need(q, "q", torch.uint8, dev)
    _need(s, "s", torch.uint8, dev)
    ld = w.stride(0) if N > 1 else K
    with torch.cuda.device(dev):
        _check(lib().mx_quantize_weight(_ptr(w), dt, N, K, ld, _ptr(q), _ptr(s), _stream(dev)))
    return q, s


def _linear_common(M, K, wq, ws, bias, y, dev):
    N = wq.shape[0]
    _need(wq, "wq", torch.uint8, dev)
    _need(ws, "ws", torch.uint8, dev)
    if wq.shape != (N, K) or ws.shape != (N, K // 32):
        raise ValueError(f"weights must be [N, {K}] codes and [N, {K // 32}] scales")
    if bias is not None:
        _need(bias, "bias", torch.float16, dev)
        if bias.shape != (N,):
            raise ValueError("bias must be f16 [N]")
    y = torch.empty((M, N), dtype=torch.bfloat16, device=dev) if y is None else y
    _need(y, "y", torch.bfloat16, dev)
    if y.shape != (M, N):
        raise ValueError("y must be bf16 [M, N]")
    return N, y


def mx_linear_fused(x, wq, ws, bias=None, gelu=False, y=None):
    """y = bf16(epi(quant_mx(x) @ dequant(wq, ws)^T + bias)) on row-major
    weights, activation quantization fused into the GEMM's prologue (slow:
    see mx.h). x: bf16 [M, K]."""
    dev = x.device
    _need(x, "x", torch.bfloat16, dev)
    M, K = x.shape
    N, y = _linear_common(M, K, wq, ws, bias, y, dev)
    epi = MX_EPI_GELU_TANH if gelu else MX_EPI_NONE
    with torch.cuda.device(dev):
        _check(lib().mx_linear_fused(_ptr(x), M, K, _ptr(wq), _ptr(ws), N, _ptr(bias), epi, _ptr(y), _stream(dev)))
    return y


def mx_linear_q(xq, xs, wq, ws, bias=None, gelu=False, y=None):
    """The same linear on pre-quantized activations xq uint8 [M, K], xs uint8 [M, K/32]."""
    dev = xq.device
    _need(xq, "xq", torch.uint8, dev)
    _need(xs, "xs", torch.uint8, dev)
    M, K = xq.shape
    if xs.shape != (M, K // 32):
        raise ValueError("xs must be [M, K/32]")
    N, y = _linear_common(M, K, wq, ws, bias, y, dev)
    epi = MX_EPI_GELU_TANH if gelu else MX_EPI_NONE
    with torch.cuda.device(dev):
        _check(
            lib().mx_linear_q(_ptr(xq), _ptr(xs), M, K, _ptr(wq), _ptr(ws), N, _ptr(bias), epi, _ptr(y), _stream(dev))
        )
    return y


class Slab(NamedTuple):
    """An operand in the slab layout: codes q uint8 [K/64, R, 64], scales s
    uint8 [K/64, R, 2], R = mx_slab_rows(rows); rows past `rows` are zero."""

    q: torch.Tensor
    s: torch.Tensor
    rows: int

    @property
    def K(self):
        return self.q.shape[0] * 64


def mx_slab_rows(rows):
    return lib().mx_slab_rows(rows)


def _slab_out(rows, K, dev, out):
    R = mx_slab_rows(rows)
    if out is None:
        return Slab(
            torch.empty((K // 64, R, 64), dtype=torch.uint8, device=dev),
            torch.empty((K // 64, R, 2), dtype=torch.uint8, device=dev),
            rows,
        )
    _need(out.q, "out.q", torch.uint8, dev)
    _need(out.s, "out.s", torch.uint8, dev)
    if out.q.shape != (K // 64, R, 64) or out.s.shape != (K // 64, R, 2) or out.rows != rows:
        raise ValueError(f"out must hold [{K // 64}, {R}, 64] codes and [{K // 64}, {R}, 2] scales for {rows} rows")
    return out


def mx_quantize_act_slab(x, out=None):
    """bf16 [M, K] (rows may be strided, K % 64 == 0) -> Slab of its MX codes and scales."""
    if x.dim() != 2 or x.dtype != torch.bfloat16 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D bf16 tensor with unit column stride")
    M, K = x.shape
    if K % 64 != 0:
        raise ValueError("the slab layout needs K % 64 == 0")
    dev = x.device
    out = _slab_out(M, K, dev, out)
    ld = x.stride(0) if M > 1 else K
    with torch.cuda.device(dev):
        _check(lib().mx_quantize_act_slab(_ptr(x), M, K, ld, _ptr(out.q), _ptr(out.s), _stream(dev)))
    return out


def mx_quantize_weight_slab(w, out=None):
    """fp32 or bf16 [N, K] (K % 64 == 0) -> Slab of its MX codes and scales."""
    if w.dim() != 2 or w.stride(1) != 1:
        raise ValueError("w must be 2-D with unit column stride")
    dt = {torch.float32: MX_DT_F32, torch.bfloat16: MX_DT_BF16}.get(w.dtype)
    if dt is None:
        raise TypeError(f"w must be float32 or bfloat16, got {w.dtype}")
    N, K = w.shape
    if K % 64 != 0:
        raise ValueError("the slab layout needs K % 64 == 0")
    dev = w.device
    out = _slab_out(N, K, dev, out)
    ld = w.stride(0) if N > 1 else K
    with torch.cuda.device(dev):
        _check(lib().mx_quantize_weight_slab(_ptr(w), dt, N, K, ld, _ptr(out.q), _ptr(out.s), _stream(dev)))
    return out


def mx_slab_pack(q, s, out=None):
    """Row-major codes uint8 [rows, K] and scales uint8 [rows, K/32] -> Slab."""
    dev = q.device
    _need(q, "q", torch.uint8, dev)
    _need(s, "s", torch.uint8, dev)
    rows, K = q.shape
    if s.shape != (rows, K // 32):
        raise ValueError("s must be [rows, K/32]")
    if K % 64 != 0:
        raise ValueError("the slab layout needs K % 64 == 0")
    out = _slab_out(rows, K, dev, out)
    with torch.cuda.device(dev):
        _check(lib().mx_slab_pack(_ptr(q), _ptr(s), rows, K, _ptr(out.q), _ptr(out.s), _stream(dev)))
    return out


def _slab_linear_args(x, w, bias):
    dev = x.q.device
    for name, t in (("x.q", x.q), ("x.s", x.s), ("w.q", w.q), ("w.s", w.s)):
        _need(t, name, torch.uint8, dev)
    M, N, K = x.rows, w.rows, x.K
    if w.K != K:
        raise ValueError(f"x has K = {K}, w has K = {w.K}")
    for name, sl in (("x", x), ("w", w)):
        R = mx_slab_rows(sl.rows)
        if sl.q.shape != (K // 64, R, 64) or sl.s.shape != (K // 64, R, 2):
            raise ValueError(f"{name} is not a slab of {sl.rows} rows and K = {K}")
    if bias is not None:
        _need(bias, "bias", torch.float16, dev)
        if bias.shape != (N,):
            raise ValueError("bias must be f16 [N]")
    return dev, M, N, K


def mx_linear_slab(x, w, bias=None, gelu=False, y=None):
    """y = bf16(epi(xhat @ what^T + bias)) on slab operands x (tokens) and w (weights)."""
    return _slab_call(lib().mx_linear_slab, x, w, bias, gelu, y)


def mx_linear_slab_m128(x, w, bias=None, gelu=False, y=None):
    """mx_linear_slab on 256 (weight rows) x 128 (tokens) tiles: the same y,
    bit for bit, with twice the tiles (for a few hundred tokens)."""
    return _slab_call(lib().mx_linear_slab_m128, x, w, bias, gelu, y)


def _slab_call(fn, x, w, bias, gelu, y):
    dev, M, N, K = _slab_linear_args(x, w, bias)
    y = torch.empty((M, N), dtype=torch.bfloat16, device=dev) if y is None else y
    _need(y, "y", torch.bfloat16, dev)
    if y.shape != (M, N):
        raise ValueError("y must be bf16 [M, N]")
    epi = MX_EPI_GELU_TANH if gelu else MX_EPI_NONE
    with torch.cuda.device(dev):
        _check(fn(_ptr(x.q), _ptr(x.s), M, K, _ptr(w.q), _ptr(w.s), N, _ptr(bias), epi, _ptr(y), _stream(dev)))
    return y


def mx_linear_slab_requant(x, w, bias=None, gelu=False, out=None):
    """The same linear returning, instead of bf16 y, the Slab of y's MX
    quantization (rows M, K = N): the next linear's activation operand."""
    dev, M, N, K = _slab_linear_args(x, w, bias)
    if N % 64 != 0:
        raise ValueError("the requantized output needs N % 64 == 0")
    out = _slab_out(M, N, dev, out)
    epi = MX_EPI_GELU_TANH if gelu else MX_EPI_NONE
    with torch.cuda.device(dev):
        _check(
            lib().mx_linear_slab_requant(
                _ptr(x.q), _ptr(x.s), M, K, _ptr(w.q), _ptr(w.s), N, _ptr(bias), epi, _ptr(out.q), _ptr(out.s),
                _stream(dev),
            )
        )
    return out


def mx_linear_splitk_ws_bytes(M, N, splits):
    return lib().mx_linear_splitk_ws_bytes(M, N, splits)


def mx_linear_splitk_choose(M, K, N):
    return lib().mx_linear_splitk_choose(M, K, N)


def mx_linear_slab_splitk(x, w, bias=None, gelu=False, y=None, splits=None, workspace=None):
    """mx_linear_slab with split-K over `splits` K ranges (default
    mx_linear_splitk_choose); workspace: uint8 of at least
    mx_linear_splitk_ws_bytes(M, N, splits) bytes (allocated here when None)."""
    dev, M, N, K = _slab_linear_args(x, w, bias)
    splits = mx_linear_splitk_choose(M, K, N) if splits is None else int(splits)
    y = torch.empty((M, N), dtype=torch.bfloat16, device=dev) if y is None else y
    _need(y, "y", torch.bfloat16, dev)
    if y.shape != (M, N):
        raise ValueError("y must be bf16 [M, N]")
    if workspace is None:
        need = mx_linear_splitk_ws_bytes(M, N, splits)
        workspace = torch.empty((max(need, 1),), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, dev)
    epi = MX_EPI_GELU_TANH if gelu else MX_EPI_NONE
    with torch.cuda.device(dev):
        _check(
            lib().mx_linear_slab_splitk(
                _ptr(x.q), _ptr(x.s), M, K, _ptr(w.q), _ptr(w.s), N, _ptr(bias), epi, _ptr(y), splits,
                _ptr(workspace), workspace.numel(), _stream(dev),
            )
        )
    return y


def mx_linear_small_ws_bytes(M, N, splits):
    return lib().mx_linear_small_ws_bytes(M, N, splits)


def mx_linear_small_choose(M, K, N):
    return lib().mx_linear_small_choose(M, K, N)


def mx_linear_slab_small(x, w, bias=None, gelu=False, y=None, splits=None, workspace=None):
    """mx_linear_slab through the few-token kernel (128 x 64 tiles) with
    `splits` K ranges (default mx_linear_small_choose); workspace: uint8 of
    at least mx_linear_small_ws_bytes(M, N, splits) bytes (allocated here
    when None and needed)."""
    dev, M, N, K = _slab_linear_args(x, w, bias)
    splits = mx_linear_small_choose(M, K, N) if splits is None else int(splits)
    y = torch.empty((M, N), dtype=torch.bfloat16, device=dev) if y is None else y
    _need(y, "y", torch.bfloat16, dev)
    if y.shape != (M, N):
        raise ValueError("y must be bf16 [M, N]")
    need = mx_linear_small_ws_bytes(M, N, splits)
    if workspace is None and need > 0:
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, dev)
    epi = MX_EPI_GELU_TANH if gelu else MX_EPI_NONE
    with torch.cuda.device(dev):
        _check(
            lib().mx_linear_slab_small(
                _ptr(x.q), _ptr(x.s), M, K, _ptr(w.q), _ptr(w.s), N, _ptr(bias), epi, _ptr(y), splits,
                _ptr(workspace), 0 if workspace is None else workspace.numel(), _stream(dev),
            )
        )
    return y


def _plan_out(fn, *args):
    kind, splits = ctypes.c_int(0), ctypes.c_int(0)
    _check(fn(*args, ctypes.byref(kind), ctypes.byref(splits)))
    return PLAN_NAMES[kind.value], splits.value


def plan_linear(M, K, N):
    """The default kernel plan of an M x K x N slab linear
    (mx_linear_plan_default): ("small", splits), ("splitk", splits) or
    ("slab", 1)."""
    return _plan_out(lib().mx_linear_plan_default, M, K, N)


def plan_lookup(M, K, N, gelu=False):
    """The tuned plan of this shape if mx_linear_tune cached one, else the
    default plan (mx_linear_plan_lookup)."""
    return _plan_out(lib().mx_linear_plan_lookup, M, K, N, MX_EPI_GELU_TANH if gelu else MX_EPI_NONE)


def plan_ws_bytes(plan, M, N, K=64):
    """Workspace bytes of a plan (mx_linear_plan_ws_bytes; K matters only to
    "balanced")."""
    kind, sp = plan
    return lib().mx_linear_plan_ws_bytes(PLAN_KINDS[kind], sp, M, K, N)


def mx_linear_tune_ws_bytes(M, K, N):
    return lib().mx_linear_tune_ws_bytes(M, K, N)


def mx_linear_plan_clear():
    lib().mx_linear_plan_clear()


def _plan_call(x, w, bias, y):
    dev, M, N, K = _slab_linear_args(x, w, bias)
    y = torch.empty((M, N), dtype=torch.bfloat16, device=dev) if y is None else y
    _need(y, "y", torch.bfloat16, dev)
    if y.shape != (M, N):
        raise ValueError("y must be bf16 [M, N]")
    return dev, M, N, K, y


def _ws_args(workspace, dev):
    if workspace is None:
        return None, 0
    _need(workspace, "workspace", torch.uint8, dev)
    return workspace, workspace.numel()


def mx_linear_slab_planned(plan, x, w, bias=None, gelu=False, y=None, workspace=None):
    """mx_linear_slab through the kernel a plan names (mx_linear_slab_plan);
    workspace: uint8 of at least plan_ws_bytes(plan, M, N, K) bytes
    (allocated here when None and needed)."""
    dev, M, N, K, y = _plan_call(x, w, bias, y)
    kind, sp = plan
    need = lib().mx_linear_plan_ws_bytes(PLAN_KINDS[kind], sp, M, K, N)
    if workspace is None and need > 0:
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
    workspace, nb = _ws_args(workspace, dev)
    epi = MX_EPI_GELU_TANH if gelu else MX_EPI_NONE
    with torch.cuda.device(dev):
        _check(lib().mx_linear_slab_plan(PLAN_KINDS[kind], sp, _ptr(x.q), _ptr(x.s), M, K, _ptr(w.q), _ptr(w.s), N,
                                         _ptr(bias), epi, _ptr(y), _ptr(workspace), nb, _stream(dev)))
    return y


def mx_linear_tune(x, w, bias=None, gelu=False, y=None, workspace=None, reps=10):
    """Times the candidate plans of this shape on these operands, caches the
    fastest (mx_linear_tune) and returns it as (kind, splits). workspace:
    uint8 of at least mx_linear_tune_ws_bytes(M, K, N) bytes (allocated here
    when None). Synchronizes the current stream."""
    dev, M, N, K, y = _plan_call(x, w, bias, y)
    if workspace is None:
        workspace = torch.empty((max(mx_linear_tune_ws_bytes(M, K, N), 1),), dtype=torch.uint8, device=dev)
    workspace, nb = _ws_args(workspace, dev)
    epi = MX_EPI_GELU_TANH if gelu else MX_EPI_NONE
    with torch.cuda.device(dev):
        return _plan_out(lib().mx_linear_tune, _ptr(x.q), _ptr(x.s), M, K, _ptr(w.q), _ptr(w.s), N, _ptr(bias), epi,
                         _ptr(y), _ptr(workspace), nb, int(reps), _stream(dev))


def mx_linear_slab_auto(x, w, bias=None, gelu=False, y=None, workspace=None):
    """mx_linear_slab through the cached (tuned) or default plan of this shape
    (mx_linear_slab_auto); workspace: uint8 of at least the plan's workspace
    (mx_linear_tune_ws_bytes always suffices; allocated here when None and
    needed)."""
    dev, M, N, K, y = _plan_call(x, w, bias, y)
    if workspace is None:
        with torch.cuda.device(dev):
            kind, sp = plan_lookup(M, K, N, gelu)
        need = lib().mx_linear_plan_ws_bytes(PLAN_KINDS[kind], sp, M, K, N)
        if need > 0:
            workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
    workspace, nb = _ws_args(workspace, dev)
    epi = MX_EPI_GELU_TANH if gelu else MX_EPI_NONE
    with torch.cuda.device(dev):
        _check(lib().mx_linear_slab_auto(_ptr(x.q), _ptr(x.s), M, K, _ptr(w.q), _ptr(w.s), N, _ptr(bias), epi,
                                         _ptr(y), _ptr(workspace), nb, _stream(dev)))
    return y


def mx_probe_mfma(a, b, iters, blocks, sink):
    """Launches the MFMA throughput probe (mx_probe_mfma) on uint8 code
    tensors a, b (same byte count, a multiple of 4) with a float32 sink of at
    least blocks * 256 elements; returns the FLOP it performs. Time it with
    events on the current stream."""
    dev = a.device
    _need(a, "a", torch.uint8, dev)
    _need(b, "b", torch.uint8, dev)
    _need(sink, "sink", torch.float32, dev)
    if a.numel() != b.numel() or sink.numel() < blocks * 256:
        raise ValueError("a and b must have equal sizes and sink at least blocks * 256 floats")
    with torch.cuda.device(dev):
        _check(lib().mx_probe_mfma(_ptr(a), _ptr(b), a.numel(), int(iters), int(blocks), _ptr(sink), _stream(dev)))
    return float(blocks) * 4 * 16 * iters * 2 * 32 * 32 * 64


def mx_linear_balanced_ws_bytes(M, K, N):
    return lib().mx_linear_balanced_ws_bytes(M, K, N)


def mx_linear_slab_balanced(x, w, bias=None, gelu=False, y=None, workspace=None):
    """mx_linear_slab with the last, partial round of tiles split over K;
    workspace: uint8 of at least mx_linear_balanced_ws_bytes(M, K, N) bytes
    (allocated here when None and needed)."""
    dev, M, N, K = _slab_linear_args(x, w, bias)
    y = torch.empty((M, N), dtype=torch.bfloat16, device=dev) if y is None else y
    _need(y, "y", torch.bfloat16, dev)
    if y.shape != (M, N):
        raise ValueError("y must be bf16 [M, N]")
    need = mx_linear_balanced_ws_bytes(M, K, N)
    if workspace is None and need > 0:
        workspace = torch.empty((need,), dtype=torch.uint8, device=dev)
    if workspace is not None:
        _need(workspace, "workspace", torch.uint8, dev)
    epi = MX_EPI_GELU_TANH if gelu else MX_EPI_NONE
    with torch.cuda.device(dev):
        _check(
            lib().mx_linear_slab_balanced(
                _ptr(x.q), _ptr(x.s), M, K, _ptr(w.q), _ptr(w.s), N, _ptr(bias), epi, _ptr(y), _ptr(workspace),
                0 if workspace is None else workspace.numel(), _stream(dev),
            )
        )
    return y


class PCSlab(NamedTuple):
    """A per-channel FP8 operand: codes q uint8 [K/64, R, 64] (slab layout)
    and one f32 scale per row s [R], R = mx_slab_rows(rows); pad rows zero."""

    q: torch.Tensor
    s: torch.Tensor
    rows: int

    @property
    def K(self):
        return self.q.shape[0] * 64


def _pc_out(rows, K, dev, out):
    R = mx_slab_rows(rows)
    if out is None:
        return PCSlab(
            torch.empty((K // 64, R, 64), dtype=torch.uint8, device=dev),
            torch.empty((R,), dtype=torch.float32, device=dev),
            rows,
        )
    _need(out.q, "out.q", torch.uint8, dev)
    _need(out.s, "out.s", torch.float32, dev)
    if out.q.shape != (K // 64, R, 64) or out.s.shape != (R,) or out.rows != rows:
        raise ValueError(f"out must hold [{K // 64}, {R}, 64] codes and [{R}] scales for {rows} rows")
    return out


def mx_pc_quantize_act_slab(x, out=None):
    """bf16 [M, K] (rows may be strided, K % 64 == 0) -> PCSlab: per-token
    FP8 codes and f32 row scales (max |x| / 448)."""
    if x.dim() != 2 or x.dtype != torch.bfloat16 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D bf16 tensor with unit column stride")
    M, K = x.shape
    if K % 64 != 0:
        raise ValueError("the slab layout needs K % 64 == 0")
    dev = x.device
    out = _pc_out(M, K, dev, out)
    ld = x.stride(0) if M > 1 else K
    with torch.cuda.device(dev):
        _check(lib().mx_pc_quantize_act_slab(_ptr(x), M, K, ld, _ptr(out.q), _ptr(out.s), _stream(dev)))
    return out


def mx_pc_quantize_weight_slab(w, out=None):
    """fp32 or bf16 [N, K] -> PCSlab: per-output-channel FP8 codes and f32 scales."""
    if w.dim() != 2 or w.stride(1) != 1:
        raise ValueError("w must be 2-D with unit column stride")
    dt = {torch.float32: MX_DT_F32, torch.bfloat16: MX_DT_BF16}.get(w.dtype)
    if dt is None:
        raise TypeError(f"w must be float32 or bfloat16, got {w.dtype}")
    N, K = w.shape
    if K % 64 != 0:
        raise ValueError("the slab layout needs K % 64 == 0")
    dev = w.device
    out = _pc_out(N, K, dev, out)
    ld = w.stride(0) if N > 1 else K
    with torch.cuda.device(dev):
        _check(lib().mx_pc_quantize_weight_slab(_ptr(w), dt, N, K, ld, _ptr(out.q), _ptr(out.s), _stream(dev)))
    return out


def mx_pc_linear_slab(x, w, bias=None, gelu=False, y=None):
    """y = bf16(epi(xs[m] ws[n] (dec(xq) @ dec(wq)^T) + bias)) on PCSlab operands."""
    dev = x.q.device
    for name, t, dt in (("x.q", x.q, torch.uint8), ("x.s", x.s, torch.float32), ("w.q", w.q, torch.uint8),
                        ("w.s", w.s, torch.float32)):
        _need(t, name, dt, dev)
    M, N, K = x.rows, w.rows, x.K
    if w.K != K:
        raise ValueError(f"x has K = {K}, w has K = {w.K}")
    for name, sl in (("x", x), ("w", w)):
        R = mx_slab_rows(sl.rows)
        if sl.q.shape != (K // 64, R, 64) or sl.s.shape != (R,):
            raise ValueError(f"{name} is not a per-channel slab of {sl.rows} rows and K = {K}")
    if bias is not None:
        _need(bias, "bias", torch.float16, dev)
        if bias.shape != (N,):
            raise ValueError("bias must be f16 [N]")
    y = torch.empty((M, N), dtype=torch.bfloat16, device=dev) if y is None else y
    _need(y, "y", torch.bfloat16, dev)
    if y.shape != (M, N):
        raise ValueError("y must be bf16 [M, N]")
    epi = MX_EPI_GELU_TANH if gelu else MX_EPI_NONE
    with torch.cuda.device(dev):
        _check(
            lib().mx_pc_linear_slab(
                _ptr(x.q), _ptr(x.s), M, K, _ptr(w.q), _ptr(w.s), N, _ptr(bias), epi, _ptr(y), _stream(dev)
            )
        )
    return y


def mx_linear_ws_bytes(M, K, N):
    return lib().mx_linear_ws_bytes(M, K, N)


def mx_linear(x, w, bias=None, gelu=False, y=None, workspace=None):
    """The linear in one call (mx.h mx_linear): bf16 x [M, K] (rows may be
    strided) is quantized into `workspace` and multiplied by the slab weights
    w through the shape's plan (tuned or default). workspace: uint8 of at
    least mx_linear_ws_bytes(M, K, N) bytes, allocated here when None."""
    if x.dim() != 2 or x.dtype != torch.bfloat16 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D bf16 tensor with unit column stride")
    dev = x.device
    M, K = x.shape
    _need(w.q, "w.q", torch.uint8, dev)
    _need(w.s, "w.s", torch.uint8, dev)
    if w.K != K:
        raise ValueError(f"x has K = {K}, w has K = {w.K}")
    N = w.rows
    if bias is not None:
        _need(bias, "bias", torch.float16, dev)
        if bias.shape != (N,):
            raise ValueError("bias must be f16 [N]")
    y = torch.empty((M, N), dtype=torch.bfloat16, device=dev) if y is None else y
    _need(y, "y", torch.bfloat16, dev)
    if y.shape != (M, N):
        raise ValueError("y must be bf16 [M, N]")
    need = mx_linear_ws_bytes(M, K, N)
    if need < 0:
        raise ValueError("the slab layout needs K % 64 == 0")
    if workspace is None:
        workspace = torch.empty((max(need, 1),), dtype=torch.uint8, device=dev)
    _need(workspace, "workspace", torch.uint8, dev)
    ld = x.stride(0) if M > 1 else K
    epi = MX_EPI_GELU_TANH if gelu else MX_EPI_NONE
    with torch.cuda.device(dev):
        _check(
            lib().mx_linear(
                _ptr(x), M, K, ld, _ptr(w.q), _ptr(w.s), N, _ptr(bias), epi, _ptr(y), _ptr(workspace),
                workspace.numel(), _stream(dev),
            )
        )
    return y


def mx_linear_noalloc(x, w, bias=None, gelu=False, y=None):
    """mx_linear with the library's own scratch array as its workspace (mx.h
    mx_linear_noalloc: no workspace argument, nothing allocated by the
    library; calls overlapping on one GPU race). y is allocated here when
    None."""
    if x.dim() != 2 or x.dtype != torch.bfloat16 or x.stride(1) != 1:
        raise ValueError("x must be a 2-D bf16 tensor with unit column stride")
    dev = x.device
    M, K = x.shape
    _need(w.q, "w.q", torch.uint8, dev)
    _need(w.s, "w.s", torch.uint8, dev)
    if w.K != K:
        raise ValueError(f"x has K = {K}, w has K = {w.K}")
    N = w.rows
    if bias is not None:
        _need(bias, "bias", torch.float16, dev)
        if bias.shape != (N,):
            raise ValueError("bias must be f16 [N]")
    y = torch.empty((M, N), dtype=torch.bfloat16, device=dev) if y is None else y
    _need(y, "y", torch.bfloat16, dev)
    if y.shape != (M, N):
        raise ValueError("y must be bf16 [M, N]")
    ld = x.stride(0) if M > 1 else K
    epi = MX_EPI_GELU_TANH if gelu else MX_EPI_NONE
    with torch.cuda.device(dev):
        _check(lib().mx_linear_noalloc(_ptr(x), M, K, ld, _ptr(w.q), _ptr(w.s), N, _ptr(bias), epi, _ptr(y),
                                       _stream(dev)))
    return y


class FP4Slab(NamedTuple):
    """An MXFP4 operand in the slab layout: codes q uint8 [S, R/16, 4, 16, 16]
    and scales s uint8 [S, R, 4], S = ceil(K/128), R = mx_slab_rows(rows);
    rows past `rows` and groups past K are zero."""

    q: torch.Tensor
    s: torch.Tensor
    rows: int
    K: int


@functools.lru_cache(maxsize=4096)
def _fp4_shapes(rows, K):
    S, R = (K + 127) // 128, (rows + 255) // 256 * 256
    return (S, R // 16, 4, 16, 16), (S, R, 4)


@functools.lru_cache(maxsize=4096)
def _fp4_ws_bytes(M, K, N, fmt):
    return lib().mx_fp4_linear_ws_bytes(M, K, N, fmt)


def _fp4_out(rows, K, like, out):
    if out is None:
        sq, ss = _fp4_shapes(rows, K)
        return FP4Slab(like.new_empty(sq, dtype=torch.uint8), like.new_empty(ss, dtype=torch.uint8), rows, K)
    _need_fp4(out, "out", like.device)
    if out.rows != rows or out.K != K:
        raise ValueError(f"out must hold {rows} rows of K = {K}")
    return out


def _need_fp4(t, name, dev):
    if not isinstance(t, FP4Slab):
        raise TypeError(f"{name} must be an FP4Slab")
    q, s, rows, K = t
    _need(q, name, torch.uint8, dev)
    _need(s, name, torch.uint8, dev)
    sq, ss = _fp4_shapes(rows, K)
    if q.shape != sq or s.shape != ss:
        raise ValueError(f"{name} is not an MXFP4 slab of {rows} rows and K = {K}")


def _act_format(act):
    if act not in ACT_FORMATS:
        raise ValueError(f"act must be 'fp8' or 'fp4', got {act!r}")
    return ACT_FORMATS[act]


def _need_rows(x, name, dtypes, shape=None, dev=None):
    """x is 2-D, of one of `dtypes`, with unit column stride (and of `shape`, on `dev`)."""
    if not isinstance(x, torch.Tensor) or x.dtype not in dtypes or x.dim() != 2:
        raise TypeError(f"{name} must be a 2-D tensor of {' or '.join(str(d) for d in dtypes)}")
    if x.stride(1) != 1 and x.shape[1] > 1:
        raise ValueError(f"{name} must have unit column stride")
    if shape is not None and (x.shape != shape or x.device != dev):
        raise ValueError(f"{name} must be {list(shape)} on {dev}")


def _pitch(x):
    return x.stride(0) if x.shape[0] > 1 else x.shape[1]


_DTYPES = {torch.float32: MX_DT_F32, torch.bfloat16: MX_DT_BF16}
_BF16 = (torch.bfloat16,)


# A call of a few tokens runs for about as long on the GPU as Python needs to
# make it, so these calls pass addresses as plain integers (None for NULL) and
# take the stream's handle without building a Stream object.


def _adr(t):
    return None if t is None else t.data_ptr()


def _run(fn, dev, *args):
    """Calls fn(*args, stream) with `dev` the current device, on its current stream."""
    i = dev.index
    if torch.cuda.current_device() == i:  # the usual case: no switch
        status = fn(*args, torch._C._cuda_getCurrentRawStream(i))
    else:
        with torch.cuda.device(dev):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(i))
    if status != MX_OK:
        _check(status)


def _fp4_quantize(x, name, dtypes, out):
    _need_rows(x, name, dtypes)
    rows, K = x.shape
    if K == 0 or K % 32 != 0:
        raise ValueError("MXFP4 needs K to be a positive multiple of 32")
    return _fp4_out(rows, K, x, out)


def mx_fp4_quantize_act_slab(x, out=None):
    """bf16 [M, K] (rows may be strided, K % 32 == 0) -> FP4Slab of its MXFP4 codes and scales."""
    out = _fp4_quantize(x, "x", (torch.bfloat16,), out)
    _run(lib().mx_fp4_quantize_act_slab, x.device, _adr(x), x.shape[0], x.shape[1], _pitch(x), _adr(out.q), _adr(out.s))
    return out


def mx_fp4_quantize_weight_slab(w, out=None):
    """fp32 or bf16 [N, K] (K % 32 == 0) -> FP4Slab of its MXFP4 codes and scales."""
    out = _fp4_quantize(w, "w", (torch.float32, torch.bfloat16), out)
    _run(lib().mx_fp4_quantize_weight_slab, w.device, _adr(w), _DTYPES[w.dtype], w.shape[0], w.shape[1], _pitch(w),
         _adr(out.q), _adr(out.s))
    return out


def mx_fp4_dequantize_slab(slab, y=None, dtype=torch.bfloat16):
    """The values of an FP4Slab as y [rows, K] (bf16 or fp32; rows may be
    strided; allocated with `dtype` when None)."""
    dev = slab.q.device
    _need_fp4(slab, "slab", dev)
    if y is None:
        if dtype not in _DTYPES:
            raise TypeError("dtype must be bfloat16 or float32")
        y = slab.q.new_empty((slab.rows, slab.K), dtype=dtype)
    else:
        _need_rows(y, "y", _DTYPES, (slab.rows, slab.K), dev)
    _run(lib().mx_fp4_dequantize_slab, dev, _adr(slab.q), _adr(slab.s), slab.rows, slab.K, _adr(y), _DTYPES[y.dtype],
         _pitch(y))
    return y


def mx_fp4_slab_pack(q, s, out=None):
    """Row-major packed codes uint8 [rows, K/2] (element 2b of a row in the
    low half of byte b) and scales uint8 [rows, K/32] -> FP4Slab."""
    dev = q.device
    _need(q, "q", torch.uint8, dev)
    _need(s, "s", torch.uint8, dev)
    if q.dim() != 2 or q.shape[1] == 0 or q.shape[1] % 16 != 0:
        raise ValueError("q must be [rows, K/2] with K a positive multiple of 32")
    rows, K = q.shape[0], 2 * q.shape[1]
    if s.shape != (rows, K // 32):
        raise ValueError("s must be [rows, K/32]")
    out = _fp4_out(rows, K, q, out)
    _run(lib().mx_fp4_slab_pack, dev, _adr(q), _adr(s), rows, K, _adr(out.q), _adr(out.s))
    return out


def mx_fp4_slab_unpack(slab, out=None):
    """An FP4Slab as the MXFP8 Slab of the same values (K % 64 == 0)."""
    dev = slab.q.device
    _need_fp4(slab, "slab", dev)
    if slab.K % 64 != 0:
        raise ValueError("the MXFP8 slab layout needs K % 64 == 0")
    out = _slab_out(slab.rows, slab.K, dev, out)
    _run(lib().mx_fp4_slab_unpack, dev, _adr(slab.q), _adr(slab.s), slab.rows, slab.K, _adr(out.q), _adr(out.s))
    return out


def _fp4_linear_out(M, w, bias, y, dev):
    _need_fp4(w, "w", dev)
    N = w.rows
    if bias is not None:
        _need(bias, "bias", torch.float16, dev)
        if bias.shape != (N,):
            raise ValueError("bias must be f16 [N]")
    if y is None:
        return w.q.new_empty((M, N), dtype=torch.bfloat16)
    _need(y, "y", torch.bfloat16, dev)
    if y.shape != (M, N):
        raise ValueError("y must be bf16 [M, N]")
    return y


def _fp4_workspace(workspace, need, dev):
    if workspace is None:
        return torch.empty((need,), dtype=torch.uint8, device=dev) if need > 0 else None
    _need(workspace, "workspace", torch.uint8, dev)
    return workspace


def mx_fp4_linear_slab(x, w, bias=None, gelu=False, y=None):
    """y = bf16(epi(xhat @ what^T + bias)) on an activation slab x (FP4Slab,
    or Slab for MXFP8 activations) and MXFP4 weights w (FP4Slab)."""
    if not isinstance(x, (FP4Slab, Slab)):
        raise TypeError("x must be an FP4Slab or a Slab")
    dev = x.q.device
    if isinstance(x, FP4Slab):
        act = "fp4"
        _need_fp4(x, "x", dev)
    else:
        act = "fp8"
        _need(x.q, "x.q", torch.uint8, dev)
        _need(x.s, "x.s", torch.uint8, dev)
        R = (x.rows + 255) // 256 * 256
        if x.q.shape != (x.K // 64, R, 64) or x.s.shape != (x.K // 64, R, 2):
            raise ValueError(f"x is not a slab of {x.rows} rows and K = {x.K}")
    M, K = x.rows, x.K
    y = _fp4_linear_out(M, w, bias, y, dev)
    if w.K != K:
        raise ValueError(f"x has K = {K}, w has K = {w.K}")
    _run(lib().mx_fp4_linear_slab, dev, ACT_FORMATS[act], _adr(x.q), _adr(x.s), M, K, _adr(w.q), _adr(w.s), w.rows,
         _adr(bias), MX_EPI_GELU_TANH if gelu else MX_EPI_NONE, _adr(y))
    return y


def mx_fp4_linear_ws_bytes(M, K, N, act="fp4"):
    return lib().mx_fp4_linear_ws_bytes(M, K, N, _act_format(act))


def mx_fp4_linear_tile(M, K, N, act="fp4"):
    """(weight rows, tokens, halved): the tiles on which mx_fp4_linear and
    mx_fp4_linear_slab compute a shape, (0, 0, False) for the few-token kernel."""
    w, t, h = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()
    _check(lib().mx_fp4_linear_tile(M, K, N, _act_format(act), ctypes.byref(w), ctypes.byref(t), ctypes.byref(h)))
    return w.value, t.value, bool(h.value)


def mx_fp4_linear(x, w, bias=None, gelu=False, act="fp4", y=None, workspace=None):
    """The linear on MXFP4 weights in one call (mx.h mx_fp4_linear): bf16 x
    [M, K] (rows may be strided) is quantized to MXFP4 (act="fp4") or MXFP8
    (act="fp8") and multiplied by the FP4Slab w. workspace: uint8 of at least
    mx_fp4_linear_ws_bytes(M, K, N, act) bytes (allocated here when None and
    needed; a few tokens need none); calls that can run at the same time, and
    graphs that captured them, need one each."""
    fmt = _act_format(act)
    _need_rows(x, "x", _BF16)
    dev = x.device
    M, K = x.shape
    y = _fp4_linear_out(M, w, bias, y, dev)
    if w.K != K:
        raise ValueError(f"x has K = {K}, w has K = {w.K}")
    workspace = _fp4_workspace(workspace, _fp4_ws_bytes(M, K, w.rows, fmt), dev)
    _run(lib().mx_fp4_linear, dev, _adr(x), M, K, _pitch(x), _adr(w.q), _adr(w.s), w.rows, _adr(bias),
         MX_EPI_GELU_TANH if gelu else MX_EPI_NONE, fmt, _adr(y), _adr(workspace),
         0 if workspace is None else workspace.numel())
    return y


def mx_rmsnorm_slab(x, weight=None, residual=None, eps=1e-6, act="fp8", out=None, residual_out=None, y=None):
    """h = x + residual, then the RMS norm of h as the activation slab of a
    quantized linear (mx.h mx_rmsnorm_slab): returns (slab, h).

    x: bf16 [M, K]; residual: bf16 or fp32 [M, K] or None; weight: bf16 or
    fp32 [K] or None (ones); rows of x, residual, residual_out and y may be
    strided. act: "fp8" gives a Slab (mx_linear_slab and its kin, and
    mx_fp4_linear_slab), "fp4" an FP4Slab. residual_out: h goes here
    (allocated when None and there is a residual; may be `residual` itself); h
    is None without a residual. y: bf16 [M, K] that also receives the norm, if
    given."""
    fmt = _act_format(act)
    _need_rows(x, "x", _BF16)
    dev, shape = x.device, x.shape
    M, K = shape
    if K == 0 or K % (32 if fmt == MX_ACT_FP4 else 64) != 0:
        raise ValueError("K must be a positive multiple of 32 (fp4) or 64 (fp8)")
    rdt = wdt = ldr = ldo = ldy = 0
    if residual is not None:
        _need_rows(residual, "residual", _DTYPES, shape, dev)
        rdt, ldr = _DTYPES[residual.dtype], _pitch(residual)
        if residual_out is None:
            residual_out = torch.empty_like(residual) if residual.is_contiguous() else residual.new_empty(shape)
            ldo = K
        else:
            _need_rows(residual_out, "residual_out", (residual.dtype,), shape, dev)
            ldo = _pitch(residual_out)
    elif residual_out is not None:
        raise ValueError("residual_out without a residual")
    if weight is not None:
        if weight.dtype not in _DTYPES:
            raise TypeError("weight must be bfloat16 or float32")
        _need(weight, "weight", weight.dtype, dev)
        if weight.shape != (K,):
            raise ValueError(f"weight must be [{K}]")
        wdt = _DTYPES[weight.dtype]
    if y is not None:
        _need_rows(y, "y", _BF16, shape, dev)
        ldy = _pitch(y)
    if fmt == MX_ACT_FP4:
        out = _fp4_out(M, K, x, out)
    elif out is None:
        R = (M + 255) // 256 * 256
        out = Slab(x.new_empty((K // 64, R, 64), dtype=torch.uint8), x.new_empty((K // 64, R, 2), dtype=torch.uint8), M)
    else:
        out = _slab_out(M, K, dev, out)
    _run(lib().mx_rmsnorm_slab, dev, x.data_ptr(), _pitch(x), _adr(residual), rdt, ldr, _adr(weight), wdt, float(eps), M, K,
         _adr(residual_out), ldo, _adr(y), ldy, fmt, out.q.data_ptr(), out.s.data_ptr())
    return out, residual_out
