"""The MXFP4-weight linears and the RMS norm where operands and outputs pass 4
GiB, on scales at their documented alignment only, and captured with what they
allocate themselves."""

import numpy as np
import pytest
import torch

import synth
from helpers import assert_linear_close, dev, f64, mx

pytestmark = pytest.mark.gpu


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


def random_fp4(rows, K, seed):
    """A slab of random codes under scales around one, pads zero."""
    g = torch.Generator(device=dev()).manual_seed(seed)
    S, R = (K + 127) // 128, (rows + 255) // 256 * 256
    q = torch.randint(0, 1 << 62, (S, R // 16, 4, 16, 2), generator=g, device=dev(), dtype=torch.int64)
    q = q.view(torch.uint8).view(S, R // 16, 4, 16, 16)
    s = torch.randint(122, 132, (S, R, 4), generator=g, device=dev(), dtype=torch.uint8)
    s[:, rows:] = 0
    for r in range(rows, R):
        q[:, r // 16, :, r % 16] = 0
    return mx().FP4Slab(q, s, rows, K)


def random_fp8(rows, K, seed):
    g = torch.Generator(device=dev()).manual_seed(seed)
    R = (rows + 255) // 256 * 256
    q = torch.randint(0, 1 << 62, (K // 64, R, 8), generator=g, device=dev(), dtype=torch.int64)
    q = (q & 0x3F3F3F3F3F3F3F3F).view(torch.uint8)  # magnitudes below 2, none NaN
    s = torch.randint(122, 132, (K // 64, R, 2), generator=g, device=dev(), dtype=torch.uint8)
    q[:, rows:] = 0
    s[:, rows:] = 0
    return mx().Slab(q, s, rows)


def last_rows(x, n):
    """The slab of x's padded rows R - n .. R - 1 (n a multiple of 256)."""
    tail = x.rows - (x.s.shape[1] - n)
    if isinstance(x, mx().FP4Slab):
        return mx().FP4Slab(x.q[:, -n // 16 :].contiguous(), x.s[:, -n:].contiguous(), tail, x.K)
    return mx().Slab(x.q[:, -n:].contiguous(), x.s[:, -n:].contiguous(), tail)


@pytest.mark.parametrize("act", ["fp4", "fp8"])
def test_output_past_4_gib(act):
    """Every output is one chain of products from the bias, whatever the tile:
    the last rows are those of a call on them alone."""
    M, K, N = 140_003, 128, 16_384
    print(f"fp4 limits: y {M}x{N} {act}", flush=True)
    x = (random_fp4 if act == "fp4" else random_fp8)(M, K, 1)
    w = random_fp4(N, K, 2)
    y = mx().mx_fp4_linear_slab(x, w)
    t = last_rows(x, 1024)
    assert same(y[-t.rows :], mx().mx_fp4_linear_slab(t, w))


@pytest.mark.parametrize("act,M", [("fp4", 560_005), ("fp8", 290_005)])
def test_tokens_past_4_gib(act, M):
    K, N = 16_384, 256
    print(f"fp4 limits: tokens {M}x{K} {act}", flush=True)
    x = (random_fp4 if act == "fp4" else random_fp8)(M, K, 3)
    assert x.q.numel() > 1 << 32
    w = random_fp4(N, K, 4)
    y = mx().mx_fp4_linear_slab(x, w)
    t = last_rows(x, 16_384)
    assert t.rows * N > 16 * 16 * 8192  # the tiled kernel too, so the same chain of products
    assert same(y[-t.rows :], mx().mx_fp4_linear_slab(t, w))


@pytest.mark.parametrize("act", ["fp4", "fp8"])
@pytest.mark.parametrize("M,K,N", [(1, 69_632, 131_072), (3, 1 << 20, 8_208), (3, 16_384, 1 << 20)])
def test_weights_past_4_gib(M, K, N, act):
    """bf16 rows, few tokens and tiles, each on the last weight rows."""
    print(f"fp4 limits: weights {N}x{K} M={M} {act}", flush=True)
    w = random_fp4(N, K, 5)
    assert w.q.numel() > 1 << 32
    x = torch.randn((M, K), generator=torch.Generator(device=dev()).manual_seed(6), device=dev()).to(torch.bfloat16)
    y = mx().mx_fp4_linear(x, w, act=act)
    t = last_rows(w, 256)
    if act == "fp4":
        xh = f64(mx().mx_fp4_dequantize_slab(mx().mx_fp4_quantize_act_slab(x), dtype=torch.float32))
    else:
        import oracle

        xh = oracle.dequantize_mx(*oracle.quantize_mx(f64(x)))
    wh = f64(mx().mx_fp4_dequantize_slab(t, dtype=torch.float32))
    assert_linear_close(y[:, -t.rows :].contiguous(), xh @ wh.T, np.abs(xh) @ np.abs(wh).T, what=f"{M}x{K}x{N} {act}")


@pytest.mark.parametrize("act", ["fp8", "fp4"])
def test_norm_past_4_gib(act):
    M, K = 540_001, 4096
    print(f"norm limits: {M}x{K} {act}", flush=True)
    d = dev()
    g = torch.Generator(device=d).manual_seed(7)
    x = torch.randn((M, K), generator=g, device=d, dtype=torch.bfloat16)
    r = torch.randn((M, K), generator=g, device=d, dtype=torch.bfloat16)
    y = torch.empty_like(x)
    slab, h = mx().mx_rmsnorm_slab(x, residual=r, act=act, y=y)
    n = M - (M + 255) // 256 * 256 + 512  # the rows of the last two blocks of 256
    y1 = torch.empty_like(y[-n:])
    s1, h1 = mx().mx_rmsnorm_slab(x[-n:], residual=r[-n:], act=act, y=y1)
    assert same(h[-n:], h1) and same(y[-n:], y1)
    if act == "fp4":
        slab = mx().FP4Slab(slab.q, slab.s, M, K)
    t = last_rows(slab, 512)
    assert torch.equal(t.q, s1.q) and torch.equal(t.s, s1.s)


@pytest.mark.parametrize("act", ["fp4", "fp8"])
@pytest.mark.parametrize("M,K,N", [(3, 640, 272), (100, 640, 528), (300, 320, 4112), (1100, 320, 4112)])
def test_scales_aligned_to_4_bytes_only(M, K, N, act):
    print(f"fp4 scale alignment M={M} {act}", flush=True)

    def shift(s):
        b = torch.empty((s.numel() + 4,), dtype=torch.uint8, device=s.device)
        v = b[4:].view(s.shape)
        v.copy_(s)
        assert v.data_ptr() % 16 == 4
        return v

    x, w = (random_fp4 if act == "fp4" else random_fp8)(M, K, 8), random_fp4(N, K, 9)
    y = mx().mx_fp4_linear_slab(x, w)
    x2 = x._replace(s=shift(x.s))
    w2 = w._replace(s=shift(w.s))
    assert same(mx().mx_fp4_linear_slab(x2, w2), y)
    assert same(mx().mx_fp4_dequantize_slab(w2), mx().mx_fp4_dequantize_slab(w))
    xb = synth.make_activation(M, K, seed=1).to(dev())
    out = mx().mx_fp4_quantize_act_slab(xb)
    again = mx().mx_fp4_quantize_act_slab(xb, out=out._replace(s=shift(torch.zeros_like(out.s))))
    assert torch.equal(again.s, out.s)


@pytest.mark.parametrize("M", [2, 150, 900])
def test_captured_with_their_own_allocations(M):
    """Two graphs of the whole chain, outputs and workspaces allocated inside the
    capture, replayed in turn and several times."""
    print(f"fp4 captured allocations M={M}", flush=True)
    d = dev()
    H, I = 512, 1088
    g1 = (1 + 0.1 * torch.randn((H,), generator=torch.Generator().manual_seed(1))).to(d)
    w1, w2 = (mx().mx_fp4_quantize_weight_slab(synth.make_weight(n, k, seed=n).to(d)) for n, k in ((I, H), (H, I)))

    def chain(x, r):
        s, h = mx().mx_rmsnorm_slab(x, g1, residual=r, act="fp4")
        u = mx().mx_fp4_linear_slab(s, w1, gelu=True)
        return mx().mx_fp4_linear(u, w2, act="fp8"), h, mx().mx_fp4_linear(u, w2, act="fp4")

    ins = [(synth.make_activation(M, H, seed=s).to(d), synth.make_activation(M, H, seed=s + 9).to(d)) for s in range(4)]
    want = [[t.clone() for t in chain(*i)] for i in ins]
    graphs = []
    for k in range(2):
        x, r = (t.clone() for t in ins[k])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            chain(x, r)
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = chain(x, r)
        graphs.append((g, x, r, out))
    for turn in range(6):
        g, x, r, out = graphs[turn % 2]
        k = (turn * 3 + 1) % 4
        x.copy_(ins[k][0])
        r.copy_(ins[k][1])
        g.replay()
        chain(*ins[(k + 1) % 4])  # eager work between replays
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(out, want[k])), turn
    del graphs
