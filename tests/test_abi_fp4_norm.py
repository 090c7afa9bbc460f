"""Host-side checks of the MXFP4 and RMS norm calls: bad arguments are
rejected before any HIP call (fake device addresses are never dereferenced),
and the Python binding rejects wrong tensors."""

import ctypes

import pytest
import torch

from helpers import mx

P = ctypes.c_void_p
OK, INV, UNS = 0, 1, 2
A, B, C, D = 0x10000000, 0x20000000, 0x30000000, 0x40000000
E, F = 0x50000000, 0x60000000


@pytest.fixture(scope="module")
def L():
    return mx().lib()


def test_quantizers_reject_bad_arguments(L):
    def qa(x=A, M=4, K=96, ld=96, q=B, s=C):
        return L.mx_fp4_quantize_act_slab(P(x), M, K, ld, P(q), P(s), P(0))

    assert qa(K=0) == INV and qa(K=48) == INV and qa(K=-32) == INV and qa(M=-1) == INV
    assert qa(K=1 << 21, ld=1 << 21) == UNS
    assert qa(ld=64) == INV and qa(ld=100) == INV  # below K; rows not 16-byte aligned
    assert qa(x=0) == INV and qa(q=0) == INV and qa(s=0) == INV
    assert qa(x=A + 2) == INV and qa(q=B + 8) == INV and qa(s=C + 2) == INV
    assert qa(q=A + 64) == INV  # codes overlap x
    assert qa(s=B + 256 * 64 - 4) == INV  # scales overlap the codes of 256 padded rows
    assert qa(M=0, x=0, q=0, s=0) == OK

    def qw(w=A, dt=1, N=4, K=32, ld=32, q=B, s=C):
        return L.mx_fp4_quantize_weight_slab(P(w), dt, N, K, ld, P(q), P(s), P(0))

    assert qw(dt=5) == INV and qw(ld=34) == INV and qw(dt=0, ld=36) == INV and qw(w=0) == INV
    assert qw(N=0, w=0, q=0, s=0) == OK

    def dq(q=B, s=C, rows=4, K=32, y=A, dt=0, ld=32):
        return L.mx_fp4_dequantize_slab(P(q), P(s), rows, K, P(y), dt, ld, P(0))

    assert dq(K=40) == INV and dq(dt=3) == INV and dq(ld=36) == INV and dq(y=0) == INV and dq(y=B + 64) == INV
    assert dq(rows=-2) == INV and dq(rows=0, q=0, s=0, y=0) == OK


def test_layout_conversions_reject_bad_arguments(L):
    def pk(q=A, s=B, rows=4, K=96, qo=C, so=D):
        return L.mx_fp4_slab_pack(P(q), P(s), rows, K, P(qo), P(so), P(0))

    assert pk(K=80) == INV and pk(rows=-1) == INV and pk(q=0) == INV and pk(so=0) == INV
    assert pk(q=A + 8) == INV and pk(qo=C + 4) == INV and pk(so=D + 1) == INV
    assert pk(qo=A) == INV and pk(so=C + 1024) == INV
    assert pk(rows=0, q=0, s=0, qo=0, so=0) == OK

    def un(q=A, s=B, rows=4, K=128, qo=C, so=D):
        return L.mx_fp4_slab_unpack(P(q), P(s), rows, K, P(qo), P(so), P(0))

    assert un(K=96) == INV  # the MXFP8 slab needs K % 64 == 0
    assert un(s=B + 2) == INV and un(so=D + 2) == INV and un(qo=0) == INV and un(qo=A + 4096) == INV
    assert un(rows=0, q=0, s=0, qo=0, so=0) == OK


def slab(act=1, xq=A, xs=B, M=8, K=96, wq=C, ws=D, N=32, bias=0, epi=0, y=E):
    return mx().lib().mx_fp4_linear_slab(act, P(xq), P(xs), M, K, P(wq), P(ws), N, P(bias), epi, P(y), P(0))


def test_linear_slab_rejects_bad_arguments():
    assert slab(act=2) == INV and slab(act=-1) == INV
    assert slab(K=40) == INV and slab(act=0, K=96) == INV  # MXFP8 activations need K % 64 == 0
    assert slab(M=-1) == INV and slab(N=-16) == INV and slab(epi=7) == INV
    assert slab(N=24) == UNS and slab(N=1 << 21) == UNS and slab(M=1 << 31) == UNS and slab(K=1 << 21) == UNS
    for name in ("xq", "xs", "wq", "ws", "y"):
        assert slab(**{name: 0}) == INV, name
    assert slab(xq=A + 8) == INV and slab(xs=B + 2) == INV and slab(wq=C + 8) == INV and slab(ws=D + 2) == INV
    assert slab(y=E + 8) == INV and slab(bias=F + 1) == INV
    assert slab(y=A + 4096) == INV and slab(y=B + 512) == INV and slab(y=C) == INV and slab(y=D + 512) == INV
    assert slab(M=0, xq=0, xs=0, wq=0, ws=0, y=0) == OK and slab(N=0, wq=0, ws=0, y=0) == OK


def one(x=A, M=40, K=96, ld=96, wq=C, ws=D, N=32, bias=0, epi=0, act=1, y=E, work=F, nb=1 << 24):
    return mx().lib().mx_fp4_linear(P(x), M, K, ld, P(wq), P(ws), N, P(bias), epi, act, P(y), P(work), nb, P(0))


def test_one_call_rejects_bad_arguments(L):
    assert one(x=0) == INV and one(x=A + 4) == INV and one(ld=88) == INV and one(ld=100) == INV
    assert one(act=3) == INV and one(act=0) == INV and one(epi=2) == INV and one(N=8) == UNS
    assert one(y=A) == INV and one(y=C + 1024) == INV
    need = L.mx_fp4_linear_ws_bytes(40, 96, 32, 1)
    assert need > 0
    assert one(nb=need - 1) == INV and one(work=0) == INV and one(work=F + 16) == INV
    assert one(work=A - 256) == INV and one(work=E) == INV and one(work=C) == INV  # overlaps x, y, the codes
    assert one(M=0, x=0, wq=0, ws=0, y=0) == OK
    f = L.mx_fp4_linear_ws_bytes
    # A few tokens ask for no workspace; long rows of them do, and so do 17.
    assert f(16, 96, 32, 1) == 0 and f(16, 6144, 32, 1) == 0 and f(16, 6176, 32, 1) > 0 and f(17, 96, 32, 1) > 0
    assert f(300, 128, 32, 1) == 512 * (64 + 4) and f(300, 128, 32, 0) == 512 * (128 + 4)
    assert f(8, 40, 32, 1) == -1 and f(-1, 96, 32, 1) == -1 and f(8, 96, -1, 1) == -1
    assert f(8, 96, 32, 0) == -1 and f(8, 96, 32, 2) == -1
    assert f(0, 96, 32, 1) == 0 and f(8, 96, 0, 1) == 0


def test_linears_refuse_too_many_tiles_before_any_launch(L):
    """2^30 x 2^20 outputs: more workgroups than a launch holds. The one-call
    linear says so before its quantizer has written to the workspace."""
    for call in (lambda: slab(M=1 << 30, N=1 << 20), lambda: one(M=1 << 30, N=1 << 20, nb=1 << 62)):
        assert call() == UNS
        assert b"tiles" in L.mx_last_error_message()


def norm(x=A, ldx=64, res=0, rdt=0, ldr=64, w=0, wdt=0, eps=1e-6, M=4, K=64, ro=0, ldo=64, y=0, ldy=64, act=0, q=B, s=C):
    return mx().lib().mx_rmsnorm_slab(P(x), ldx, P(res), rdt, ldr, P(w), wdt, eps, M, K, P(ro), ldo, P(y), ldy, act, P(q),
                                      P(s), P(0))


def test_rmsnorm_rejects_bad_arguments():
    assert norm(act=5) == INV and norm(K=96) == INV and norm(act=1, K=48) == INV
    assert norm(K=65536 + 64, ldx=1 << 17) == UNS and norm(M=(1 << 22) + 1) == UNS and norm(M=-1) == INV
    assert norm(eps=-1.0) == INV and norm(eps=float("nan")) == INV and norm(eps=float("inf")) == INV
    assert norm(res=D, rdt=2) == INV and norm(w=D, wdt=9) == INV
    assert norm(ro=E) == INV  # residual_out without a residual
    assert norm(ldx=32) == INV and norm(ldx=68) == INV
    assert norm(res=D, ldr=68) == INV and norm(res=D, rdt=1, ldr=66) == INV and norm(res=D, ldr=32) == INV
    assert norm(res=D, ro=E, ldo=68) == INV and norm(y=E, ldy=32) == INV
    assert norm(x=0) == INV and norm(q=0) == INV and norm(s=0) == INV
    assert norm(x=A + 2) == INV and norm(res=D + 8) == INV and norm(w=D + 2) == INV and norm(y=E + 4) == INV
    assert norm(q=B + 8) == INV and norm(s=C + 4) == INV
    assert norm(q=A) == INV and norm(y=A + 128) == INV and norm(s=B + 1024) == INV
    assert norm(res=D, ro=D + 128) == INV  # in place means the very same rows
    assert norm(res=D, ro=D, ldr=64, ldo=72) == INV
    assert norm(res=D, ro=A) == INV and norm(res=D, ro=E, y=E + 128) == INV
    assert norm(M=0, x=0, q=0, s=0) == OK


def test_rmsnorm_takes_any_finite_eps():
    assert all(norm(eps=e, M=0, x=0, q=0, s=0) == OK for e in (0.0, 1e-300, 1.0, 1e31, 1e300))


def test_binding_rejects_wrong_tensors():
    m = mx()
    with pytest.raises(TypeError):
        m.mx_fp4_quantize_act_slab(torch.zeros(4, 64))
    with pytest.raises(TypeError):
        m.mx_fp4_quantize_weight_slab(torch.zeros(4, 64, dtype=torch.float16))
    with pytest.raises(ValueError):
        m.mx_fp4_quantize_weight_slab(torch.zeros(4, 48))
    with pytest.raises(ValueError):
        m.mx_fp4_quantize_weight_slab(torch.zeros(64, 4).t())
    w = m.FP4Slab(torch.zeros(1, 16, 4, 16, 16, dtype=torch.uint8), torch.zeros(1, 256, 4, dtype=torch.uint8), 16, 64)
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        m.mx_fp4_linear(x, w, act="fp6")
    with pytest.raises(ValueError):
        m.mx_fp4_linear(torch.zeros(4, 96, dtype=torch.bfloat16), w)
    with pytest.raises(TypeError):
        m.mx_fp4_linear(x, m.Slab(w.q, w.s, 16))
    with pytest.raises(ValueError):
        m.mx_fp4_linear(x, m.FP4Slab(w.q, w.s, 300, 64))
    with pytest.raises(TypeError):
        m.mx_fp4_linear(x, w, bias=torch.zeros(16))
    with pytest.raises(TypeError):
        m.mx_fp4_linear_slab(x, w)
    with pytest.raises(ValueError):
        m.mx_fp4_slab_unpack(m.FP4Slab(w.q, w.s, 16, 96))
    with pytest.raises(ValueError):
        m.mx_rmsnorm_slab(x, residual_out=x)
    with pytest.raises(ValueError):
        m.mx_rmsnorm_slab(x, residual=torch.zeros(5, 64, dtype=torch.bfloat16))
    with pytest.raises(TypeError):
        m.mx_rmsnorm_slab(x, residual=torch.zeros(4, 64, dtype=torch.float16))
    with pytest.raises(ValueError):
        m.mx_rmsnorm_slab(x, weight=torch.zeros(63))
