"""Host-side checks of routing, the experts' products and the block norm: bad
arguments are rejected before any HIP call (fake device addresses are never
dereferenced), and the Python binding rejects wrong tensors."""

import ctypes

import pytest
import torch

from helpers import mx

P = ctypes.c_void_p
D = ctypes.c_double
OK, INV, UNS = 0, 1, 2
A, B, C, F, G, H, J, K_ = (i << 40 for i in range(1, 9))
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def L():
    return mx().lib()


def test_route_rejects_bad_arguments(L):
    def r(logits=A, dt=1, T=4, E=16, ld=16, bias=0, scores=0, groups=1, top=1, k=2, renorm=1, scale=1.0, ids=B, w=C):
        return L.mx_route(P(logits), dt, T, E, ld, P(bias), scores, groups, top, k, renorm, D(scale), P(ids), P(w), P(0))

    assert r(T=-1) == INV and r(dt=2) == INV and r(scores=2) == INV and r(E=0) == INV and r(ld=15) == INV
    assert r(groups=0) == INV and r(groups=3) == INV and r(groups=4, top=5) == INV and r(top=0) == INV
    assert r(k=0) == INV and r(k=17) == INV and r(groups=4, top=1, k=5) == INV
    assert r(scale=INF) == INV and r(scale=NAN) == INV
    assert r(E=1025, ld=1025) == UNS and r(E=128, ld=128, k=65) == UNS and r(E=130, ld=130, groups=65, top=65) == UNS
    assert r(T=(1 << 26) + 1) == UNS
    assert r(logits=0) == INV and r(ids=0) == INV and r(w=0) == INV
    assert r(logits=A + 2) == INV and r(bias=F + 2) == INV and r(ids=B + 2) == INV and r(w=C + 1) == INV
    assert r(ids=A + 4 * 16 * 3) == INV and r(w=A) == INV and r(ids=C + 28) == INV  # overlaps
    assert r(bias=B + 4) == INV and r(bias=C) == INV
    assert r(T=0, logits=0, ids=0, w=0) == OK


def experts(L, x=A, T=5, H_=64, ldx=64, ids=B, w=C, k=2, uq=F, us=G, dq=H, ds=J, E=3, I=32, gate=0, act=0, y=K_, ws=K_ * 2,
            nb=1 << 40):
    return L.mx_fp4_experts(P(x), T, H_, ldx, P(ids), P(w), k, P(uq), P(us), P(dq), P(ds), E, I, gate, act, P(y), P(ws), nb,
                            P(0))


def test_experts_reject_bad_arguments(L):
    def e(**kw):
        return experts(L, **kw)

    assert e(T=-1) == INV and e(H_=48, ldx=48) == INV and e(I=16) == INV and e(H_=0) == INV and e(I=-32) == INV
    assert e(k=0) == INV and e(E=0) == INV and e(gate=2) == INV and e(act=2) == INV
    assert e(ldx=56) == INV and e(ldx=65) == INV
    assert e(H_=65568, ldx=65568) == UNS and e(I=65568) == UNS and e(k=65) == UNS and e(E=1025) == UNS
    assert e(T=1 << 20, k=32) == UNS  # pairs
    assert e(T=1 << 18, H_=8192, ldx=8192, k=1) == UNS  # T H
    assert e(T=1 << 18, k=64, I=16384) == UNS  # (2^17 + 3) * 2 * 128 workgroups
    for name in ("x", "ids", "w", "uq", "us", "dq", "ds", "y", "ws"):
        assert e(**{name: 0}) == INV, name
    for name, off in (("x", 8), ("uq", 8), ("dq", 4), ("y", 8), ("ids", 2), ("w", 1), ("us", 2), ("ds", 1), ("ws", 128)):
        base = {"x": A, "ids": B, "w": C, "uq": F, "us": G, "dq": H, "ds": J, "y": K_, "ws": K_ * 2}[name]
        assert e(**{name: base + off}) == INV, name
    need = L.mx_fp4_experts_ws_bytes(5, 2, 3, 64, 32, 0)
    assert need > 0 and e(nb=need - 1) == INV
    for name in ("x", "ids", "w", "uq", "us", "dq", "ds"):
        base = {"x": A, "ids": B, "w": C, "uq": F, "us": G, "dq": H, "ds": J}[name]
        assert e(y=base) == INV and e(ws=base) == INV, name
    assert e(ws=K_) == INV
    assert e(T=0, x=0, ids=0, w=0, uq=0, us=0, dq=0, ds=0, y=0, ws=0, nb=0) == OK


def test_experts_workspace_bytes(L):
    f = L.mx_fp4_experts_ws_bytes
    assert f(0, 2, 3, 64, 32, 0) == 0
    assert f(5, 2, 3, 64, 48, 0) == -1 and f(-1, 2, 3, 64, 32, 0) == -1 and f(5, 2, 3, 64, 32, 3) == -1
    assert f(5, 0, 3, 64, 32, 1) == -1 and f(5, 2, 0, 64, 32, 1) == -1
    assert f(64, 4, 8, 512, 256, 1) < f(64, 4, 8, 512, 256, 0) < f(128, 4, 8, 512, 256, 0)
    assert f(64, 4, 8, 512, 256, 0) % 256 == 0


def norm(L, x=A, ldx=128, r=B, rdt=0, ldr=128, alpha=1.0, post=0, pw=0, gate=0, grows=1, ldg=128, kind=0, w=0, sc=0, sh=0,
         mrows=1, ldm=128, vdt=1, eps=1e-6, M=6, K=128, ro=C, ldo=128, y=0, ldy=128, act=0, q=F, s=G):
    return L.mx_block_norm_slab(P(x), ldx, P(r), rdt, ldr, D(alpha), post, P(pw), P(gate), grows, ldg, kind, P(w), P(sc),
                                P(sh), mrows, ldm, vdt, D(eps), M, K, P(ro), ldo, P(y), ldy, act, P(q), P(s), P(0))


def test_block_norm_rejects_bad_arguments(L):
    def n(**kw):
        return norm(L, **kw)

    assert n(M=-1) == INV and n(K=0) == INV and n(K=96, act=0) == INV and n(K=48, act=1) == INV and n(act=2) == INV
    assert n(K=65600, ldx=65600, ldr=65600, ldo=65600) == UNS and n(M=(1 << 22) + 1) == UNS
    assert n(eps=-1.0) == INV and n(eps=NAN) == INV and n(alpha=INF) == INV and n(alpha=1e300) == INV
    assert n(rdt=2) == INV and n(w=H, vdt=2) == INV and n(kind=2) == INV and n(pw=H, post=0) == INV
    assert n(ldx=120) == INV and n(ldx=132) == INV and n(ldr=120) == INV and n(rdt=1, ldr=130) == INV
    assert n(ldo=64) == INV and n(y=H, ldy=100) == INV and n(y=H, ldy=129) == INV
    assert n(gate=H, grows=0) == INV and n(gate=H, grows=4) == INV and n(gate=H, ldg=64) == INV and n(gate=H, ldg=129) == INV
    assert n(sc=H, mrows=5) == INV and n(sh=H, mrows=0) == INV and n(sh=H, ldm=126) == INV
    assert n(x=0) == INV and n(r=0) == INV and n(q=0) == INV and n(s=0) == INV and n(q=0, s=0) == INV
    for name in ("x", "r", "ro", "q", "s"):
        base = {"x": A, "r": B, "ro": C, "q": F, "s": G}[name]
        assert n(**{name: base + 8}) == INV, name
    for name in ("pw", "gate", "w", "sc", "sh", "y"):
        assert n(post=1, **{name: H + 8}) == INV, name
    # overlaps: outputs with inputs and with each other
    assert n(ro=A) == INV and n(ro=B, ldo=136) == INV and n(ro=B + 16) == INV and n(q=A) == INV and n(s=B) == INV
    assert n(y=A) == INV and n(y=C) == INV and n(q=G) == INV and n(ro=F) == INV
    for name in ("pw", "gate", "w", "sc", "sh"):
        assert n(post=1, y=H, **{name: H}) == INV, name
    assert n(M=0, x=0, r=0, ro=0, q=0, s=0) == OK and n(M=0, x=0, r=0, ro=0, q=0, s=0, y=0, gate=H, grows=3) == OK


def test_python_binding_rejects_wrong_tensors():
    m = mx()
    lg = torch.zeros((4, 8))
    for bad in (lambda: m.mx_route(lg, 2, scores="relu"), lambda: m.mx_route(lg[0], 2), lambda: m.mx_route(lg.half(), 2),
                lambda: m.mx_route(lg.t(), 2), lambda: m.mx_route(lg, 0), lambda: m.mx_route(lg, 2, bias=torch.zeros(7)),
                lambda: m.mx_route(lg, 2, bias=torch.zeros(8).double()),
                lambda: m.mx_route(lg, 2, ids=torch.zeros((4, 2), dtype=torch.int64)),
                lambda: m.mx_route(lg, 2, weights=torch.zeros((4, 3)))):
        with pytest.raises((TypeError, ValueError)):
            bad()

    def ex(E, N, K):
        S, R = (K + 127) // 128, (N + 255) // 256 * 256
        return m.FP4Experts(torch.zeros((E, S, R // 16, 4, 16, 16), dtype=torch.uint8),
                            torch.zeros((E, S, R, 4), dtype=torch.uint8), N, K)

    x, ids, w = torch.zeros((3, 64)).bfloat16(), torch.zeros((3, 2), dtype=torch.int32), torch.zeros((3, 2))
    up, down = ex(4, 64, 64), ex(4, 64, 32)
    f = m.mx_fp4_experts
    for bad in (lambda: f(x, ids, w, up, down, gate="relu"), lambda: f(x, ids, w, up, down, act="fp16"),
                lambda: f(x.float(), ids, w, up, down), lambda: f(x, ids.long(), w, up, down),
                lambda: f(x, ids, w.double(), up, down), lambda: f(x, ids[:2], w, up, down),
                lambda: f(x, ids, w[:, :1].contiguous(), up, down), lambda: f(x, ids, w, ex(4, 64, 96), down),
                lambda: f(x, ids, w, ex(4, 128, 64), down), lambda: f(x, ids, w, up, ex(3, 64, 32)),
                lambda: f(x, ids, w, up, ex(4, 96, 32)), lambda: f(x, ids, w, up._replace(rows=32), down),
                lambda: f(x, ids, w, up.q, down), lambda: f(x, ids, w, up, down, y=torch.zeros((3, 32)).bfloat16()),
                lambda: f(x, ids, w, up, down, workspace=torch.zeros(8))):
        with pytest.raises((TypeError, ValueError)):
            bad()
    for bad in (lambda: m.mx_fp4_quantize_experts(torch.zeros((4, 64))),
                lambda: m.mx_fp4_quantize_experts(torch.zeros((2, 4, 48))),
                lambda: m.mx_fp4_quantize_experts(torch.zeros((4, 64, 32)), out=up)):
        with pytest.raises((TypeError, ValueError)):
            bad()

    r, v = torch.zeros((3, 64)).bfloat16(), torch.zeros(64)
    g = m.mx_block_norm_slab
    for bad in (lambda: g(x, r, kind="batch"), lambda: g(x, r, act="fp16"), lambda: g(x, r[:2]), lambda: g(x, r.half()),
                lambda: g(x.float(), r), lambda: g(x[:, :32], r[:, :32]), lambda: g(x, r, weight=v, gate=v.bfloat16()),
                lambda: g(x, r, weight=v.half()), lambda: g(x, r, weight=v[:32]), lambda: g(x, r, weight=v[None]),
                lambda: g(x, r, gate=torch.zeros((2, 64))), lambda: g(x, r, scale=v, shift=torch.zeros((3, 64))),
                lambda: g(x, r, residual_out=r.float()), lambda: g(x, r, y=r[:2]), lambda: g(x, r, act=None, out=r),
                lambda: g(x, r, gate=torch.zeros((0, 64))), lambda: g(x, r, gate=torch.zeros((64, 3)).t())):
        with pytest.raises((TypeError, ValueError)):
            bad()
