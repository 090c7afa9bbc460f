"""GPU parity of the MXFP4-weight linears against the oracle in float64, on
every route of the calls (bf16 rows quantized in the kernel, slab operands,
few and many tokens), with MXFP4 and MXFP8 activations.

Tolerance: the library's for every linear, 1e-3 g S + one bf16 ulp with
S = sum |xhat| |what| and g the epilogue's largest slope (oracle.tolerance):
products are exact, each MFMA adds 128 (or 64) of them with at most 2^-12 of
their absolute sum lost to alignment (mixed and FP8 operands; E2M1 products
lose none of it), the at most K / 64 + 8 fp32 additions lose 2^-24 of S each,
and the output's rounding half an ulp."""

import numpy as np
import pytest
import torch

import oracle
import synth
from helpers import assert_linear_close, dev, f64, mx

pytestmark = pytest.mark.gpu


def reference(x, w, b, act, gelu):
    xh = oracle.dequantize_fp4(*oracle.quantize_fp4(f64(x))) if act == "fp4" else oracle.dequantize_mx(
        *oracle.quantize_mx(f64(x)))
    wh = oracle.dequantize_fp4(*oracle.quantize_fp4(f64(w)))
    return oracle.linear_values_ref(xh, wh, None if b is None else f64(b), "gelu_tanh" if gelu else "none")


def quantized(x, act):
    return mx().mx_fp4_quantize_act_slab(x) if act == "fp4" else mx().mx_quantize_act_slab(x)


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


CASES = [
    (1, 32, 16), (1, 5120, 272), (2, 96, 48), (7, 1088, 256), (15, 160, 512), (16, 2048, 16), (17, 1024, 80),
    (31, 4128, 96), (33, 64, 1040), (64, 608, 304), (65, 256, 256), (100, 3200, 528), (129, 128, 64), (257, 1216, 272),
    (300, 352, 2064), (513, 544, 528), (1025, 192, 784),
    # every tile shape of the few-token kernel, and long rows of a few tokens
    (16, 6208, 5136), (3, 8256, 4112), (32, 128, 5136), (30, 320, 16400), (64, 160, 4112), (63, 96, 12304),
    (130, 96, 6160), (250, 12352, 4368), (16, 32, 20496), (10, 13824, 48), (1, 8320, 5136),
    # every shape of the tiled kernel: one step, an odd and an even number,
    # more and fewer than the ring; ragged rows, columns and K
    (260, 96, 4112), (700, 1184, 2320), (513, 544, 8208), (1000, 416, 5136), (520, 64, 10224), (1500, 288, 4112),
    (2100, 416, 5136), (4111, 64, 2576), (4000, 1184, 4368), (3100, 320, 8240),
]


@pytest.mark.parametrize("act", ["fp4", "fp8"])
@pytest.mark.parametrize("M,K,N", CASES)
def test_linear_matches_oracle(M, K, N, act):
    if act == "fp8":
        K = (K + 63) // 64 * 64
    print(f"fp4 linear M={M} K={K} N={N} {act}", flush=True)
    d = dev()
    gelu = (M + N // 16) % 2 == 1
    x = synth.make_activation(M, K, seed=M)
    w = synth.make_weight(N, K, seed=N) * 4
    b = None if M % 5 == 0 else synth.make_bias(N, seed=K)
    ws = mx().mx_fp4_quantize_weight_slab(w.to(d))
    bd = None if b is None else b.to(d)
    # Rows of x and y inside larger buffers; every element of y written, none
    # past its end.
    xb = torch.full((M, K + 8), float("nan"), dtype=torch.bfloat16, device=d)
    xb[:, :K] = x.to(d)
    yb = torch.full((M * N + 4096,), -1, dtype=torch.int16, device=d)
    y = yb[: M * N].view(torch.bfloat16).view(M, N)
    mx().mx_fp4_linear(xb[:, :K], ws, bd, gelu=gelu, act=act, y=y)
    torch.cuda.synchronize()
    assert bool((yb[M * N :] == -1).all()), "wrote past the end of y"
    assert not bool((yb[: M * N] == -1).any()), "elements of y left unwritten"
    ref, S = reference(x, w, b, act, gelu)
    assert_linear_close(y, ref, S, "gelu_tanh" if gelu else "none", what=f"{M}x{K}x{N} {act}")
    # The slab call gives the same bits, whatever the workspace held.
    ys = mx().mx_fp4_linear_slab(quantized(x.to(d), act), ws, bd, gelu=gelu)
    assert same(ys, y)


@pytest.mark.parametrize("act,M,K,N", [
    ("fp4", 17, 96, 2160), ("fp4", 18, 96, 6160), ("fp4", 17, 96, 4160), ("fp4", 17, 96, 8480), ("fp4", 33, 96, 4112),
    ("fp4", 33, 96, 6304), ("fp4", 34, 96, 8352), ("fp4", 49, 96, 10320), ("fp4", 50, 96, 8224), ("fp4", 65, 2080, 9616),
    ("fp4", 66, 4128, 10976), ("fp4", 65, 2080, 8240),
    ("fp8", 17, 64, 2192), ("fp8", 146, 64, 1616), ("fp8", 17, 192, 4240), ("fp8", 17, 192, 8224), ("fp8", 17, 64, 6160),
    ("fp8", 17, 192, 12368), ("fp8", 33, 64, 10896), ("fp8", 97, 192, 7216), ("fp8", 33, 192, 6464),
    ("fp8", 33, 64, 8368), ("fp8", 98, 1152, 8224), ("fp8", 65, 2112, 10960), ("fp8", 49, 64, 10352),
    ("fp8", 65, 4160, 13808),
])
def test_every_few_token_tile(act, M, K, N):
    """Each shape of the few-token kernel's tiles, at sizes that it does not divide."""
    print(f"fp4 few-token tile M={M} K={K} N={N} {act}", flush=True)
    d = dev()
    gelu = M % 2 == 0
    x = synth.make_activation(M, K, seed=M)
    w = synth.make_weight(N, K, seed=N) * 4
    b = synth.make_bias(N, seed=K)
    y = mx().mx_fp4_linear(x.to(d), mx().mx_fp4_quantize_weight_slab(w.to(d)), b.to(d), gelu=gelu, act=act)
    ref, S = reference(x, w, b, act, gelu)
    assert_linear_close(y, ref, S, "gelu_tanh" if gelu else "none", what=f"{M}x{K}x{N} {act}")


@pytest.mark.parametrize("act,M,K,N", [
    ("fp4", 2310, 96, 7184), ("fp4", 2561, 416, 7184), ("fp4", 4400, 160, 4112), ("fp4", 8300, 672, 2320),
    ("fp8", 1100, 192, 8208), ("fp8", 1281, 448, 7440), ("fp8", 2100, 64, 5136), ("fp8", 6000, 320, 2832),
])
def test_halved_last_round(act, M, K, N):
    """A last round of at most half the tiles behind whole ones runs in halves:
    halves that are empty or ragged, one whole round and two."""
    print(f"fp4 halved M={M} K={K} N={N} {act}", flush=True)
    d = dev()
    gelu = M % 4 == 0
    x = synth.make_activation(M, K, seed=M)
    w = synth.make_weight(N, K, seed=N) * 4
    b = synth.make_bias(N, seed=K)
    yb = torch.full((M * N + 4096,), -1, dtype=torch.int16, device=d)
    y = yb[: M * N].view(torch.bfloat16).view(M, N)
    mx().mx_fp4_linear(x.to(d), mx().mx_fp4_quantize_weight_slab(w.to(d)), b.to(d), gelu=gelu, act=act, y=y)
    assert bool((yb[M * N :] == -1).all()) and not bool((yb[: M * N] == -1).any())
    ref, S = reference(x, w, b, act, gelu)
    assert_linear_close(y, ref, S, "gelu_tanh" if gelu else "none", what=f"{M}x{K}x{N} {act}")


@pytest.mark.parametrize("K", [96, 256, 352, 512, 640, 736, 896, 1024, 1120, 1920, 2048, 2144, 3168])
def test_every_remainder_of_steps_on_small_tiles(K):
    """The 128 x 128 tiles run steps of 128 K in blocks of eight: every remainder,
    less than a block, one, more; ragged rows and columns, with and without GELU."""
    M, N = 699, 2320
    gelu = K % 256 == 0
    print(f"fp4 small tiles K={K}", flush=True)
    d = dev()
    x = synth.make_activation(M, K, seed=K)
    w = synth.make_weight(N, K, seed=K + 1) * 4
    b = synth.make_bias(N, seed=K) if K % 3 else None
    y = mx().mx_fp4_linear(x.to(d), mx().mx_fp4_quantize_weight_slab(w.to(d)), None if b is None else b.to(d), gelu=gelu)
    ref, S = reference(x, w, b, "fp4", gelu)
    assert_linear_close(y, ref, S, "gelu_tanh" if gelu else "none", what=f"K={K}")


@pytest.mark.parametrize("act", ["fp4", "fp8"])
@pytest.mark.parametrize("M,K,N", [(1, 5120, 5136), (16, 4096, 2064), (7, 8256, 4112), (5, 13824, 6160), (11, 8832, 1040),
                                   (9, 8192, 16400)])
def test_one_call_sums_in_the_slab_calls_order(M, K, N, act):
    """Products that cancel: the second half of K holds the first's groups in
    another order with the weights negated, and the groups span many binades,
    so that what is left is the fp32 sums' rounding, which shows the order of
    the sums. The one-call linear, which quantizes a few tokens in its kernel,
    adds in the slab call's order."""
    print(f"fp4 order M={M} K={K} N={N} {act}", flush=True)
    d = dev()
    g = torch.Generator(device=d).manual_seed(M + K)
    n = K // 64  # groups in a half
    x = torch.randn((M, n, 32), generator=g, device=d) * torch.exp2(8 * torch.randn((1, n, 1), generator=g, device=d))
    w = torch.randn((N, n, 32), generator=g, device=d)
    order = torch.randperm(n, generator=g, device=d)
    x = torch.cat([x, x[:, order]], 1).reshape(M, K).to(torch.bfloat16)
    ws = mx().mx_fp4_quantize_weight_slab(torch.cat([w, -w[:, order]], 1).reshape(N, K))
    y = mx().mx_fp4_linear(x, ws, act=act)
    assert bool((y != 0).any())
    assert same(mx().mx_fp4_linear_slab(quantized(x, act), ws), y)


@pytest.mark.parametrize("act", ["fp4", "fp8"])
@pytest.mark.parametrize("M", [1, 13, 40, 300, 700])
def test_rows_are_independent_of_their_batch(M, act):
    """A token's output does not change with the tokens behind it, as long as
    the call takes the same kernel."""
    print(f"fp4 rows M={M} {act}", flush=True)
    d = dev()
    K, N = 640, 272
    x = synth.make_activation(M, K, seed=M).to(d)
    w = mx().mx_fp4_quantize_weight_slab(synth.make_weight(N, K, seed=1).to(d))
    y = mx().mx_fp4_linear(x, w, act=act)
    z = x.clone()
    z[M // 2 :] = float("nan")
    yz = mx().mx_fp4_linear(z, w, act=act)
    assert same(yz[: M // 2], y[: M // 2])
    assert bool(torch.isnan(yz[M // 2 :]).all())


@pytest.mark.parametrize("act", ["fp4", "fp8"])
@pytest.mark.parametrize("M", [3, 50, 600])
def test_nonfinite_groups(M, act):
    """A NaN or Inf in a token's group makes that token's outputs NaN; one in a
    weight row's group makes that output column NaN; nothing else changes."""
    print(f"fp4 nonfinite M={M} {act}", flush=True)
    d = dev()
    K, N = 320, 272
    x = synth.make_activation(M, K, seed=2)
    w = synth.make_weight(N, K, seed=3)
    clean = mx().mx_fp4_linear(x.to(d), mx().mx_fp4_quantize_weight_slab(w.to(d)), act=act)
    x[1, 200] = float("inf")
    x[M - 1, 0] = float("nan")
    w[5, 319] = float("nan")
    w[N - 1, 64] = -float("inf")
    y = mx().mx_fp4_linear(x.to(d), mx().mx_fp4_quantize_weight_slab(w.to(d)), act=act)
    want = torch.zeros((M, N), dtype=torch.bool)
    want[1] = want[M - 1] = True
    want[:, 5] = want[:, N - 1] = True
    assert torch.equal(torch.isnan(y).cpu(), want)
    keep = (~want).to(d)
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("act", ["fp4", "fp8"])
@pytest.mark.parametrize("M", [4, 90, 1100])
def test_graph_replays_match_eager(M, act):
    print(f"fp4 graph M={M} {act}", flush=True)
    d = dev()
    K, N = 576, 528
    w = mx().mx_fp4_quantize_weight_slab(synth.make_weight(N, K, seed=4).to(d))
    ins = [synth.make_activation(M, K, seed=s).to(d) for s in (1, 2, 3)]
    x = ins[0].clone()
    res = torch.randn((M, K), device=d).to(torch.bfloat16)
    y = torch.empty((M, N), dtype=torch.bfloat16, device=d)
    y2 = torch.empty_like(y)
    ws = torch.empty((max(mx().mx_fp4_linear_ws_bytes(M, K, N, act), 1),), dtype=torch.uint8, device=d)
    h = torch.empty_like(res)
    slab, _ = mx().mx_rmsnorm_slab(x, residual=res, residual_out=h, act=act)

    def step():
        mx().mx_fp4_linear(x, w, act=act, y=y, workspace=ws)
        mx().mx_rmsnorm_slab(x, residual=res, residual_out=h, act=act, out=slab)
        mx().mx_fp4_linear_slab(slab, w, gelu=True, y=y2)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for xin in ins + ins[:1]:
        x.copy_(xin)
        ws.fill_(0xFF)
        g.replay()
        torch.cuda.synchronize()
        a, b = y.clone(), y2.clone()
        step()
        torch.cuda.synchronize()
        assert same(a, y) and same(b, y2)
    del g


@pytest.mark.parametrize("act", ["fp4", "fp8"])
def test_two_streams_at_once(act):
    """Calls on two streams with their own workspaces do not meet."""
    print(f"fp4 two streams {act}", flush=True)
    d = dev()
    K, N = 2048, 1024
    w = mx().mx_fp4_quantize_weight_slab(synth.make_weight(N, K, seed=4).to(d))
    xs = [synth.make_activation(m, K, seed=m).to(d) for m in (130, 700)]
    want = [mx().mx_fp4_linear(x, w, act=act) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [[], []]
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(mx().mx_fp4_linear(xs[i], w, act=act))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(same(y, want[i]) for y in got[i])


@pytest.mark.parametrize("M", [2, 200])
def test_block_of_norm_projection_and_feed_forward(M):
    """The operators as a serving block runs them: norm (MXFP8) -> W4A8
    projection -> residual add and norm (MXFP4) -> W4A4 up-projection with GELU
    -> W4A8 down-projection, each step against the oracle on the values that
    the step before produced."""
    print(f"fp4 block M={M}", flush=True)
    d = dev()
    H, I = 320, 704
    x = synth.make_activation(M, H, seed=1)
    r = (2 * torch.randn((M, H), generator=torch.Generator().manual_seed(2))).to(torch.bfloat16)
    g1 = 1 + 0.1 * torch.randn((H,), generator=torch.Generator().manual_seed(3))
    w = [synth.make_weight(n, k, seed=n + k) * 4 for n, k in ((H, H), (I, H), (H, I))]
    b = [synth.make_bias(n, seed=n) for n in (H, I, H)]
    wd = [mx().mx_fp4_quantize_weight_slab(t.to(d)) for t in w]
    wh = [oracle.dequantize_fp4(*oracle.quantize_fp4(f64(t))) for t in w]
    s1, h1 = mx().mx_rmsnorm_slab(x.to(d), g1.to(d), residual=r.to(d))
    y1 = mx().mx_fp4_linear_slab(s1, wd[0], b[0].to(d))
    s2, h2 = mx().mx_rmsnorm_slab(y1, residual=h1, act="fp4")
    y2 = mx().mx_fp4_linear_slab(s2, wd[1], b[1].to(d), gelu=True)
    y3 = mx().mx_fp4_linear(y2, wd[2], b[2].to(d), act="fp8")
    rh1, n1 = oracle.rmsnorm_ref(f64(x), f64(r), f64(g1))
    assert np.array_equal(f64(h1), rh1)
    ref, S = oracle.linear_values_ref(oracle.dequantize_mx(*oracle.quantize_mx(n1)), wh[0], f64(b[0]))
    assert_linear_close(y1, ref, S, what="projection")
    rh2, n2 = oracle.rmsnorm_ref(f64(y1), f64(h1))
    assert np.array_equal(f64(h2), rh2)
    ref, S = oracle.linear_values_ref(oracle.dequantize_fp4(*oracle.quantize_fp4(n2)), wh[1], f64(b[1]), "gelu_tanh")
    assert_linear_close(y2, ref, S, "gelu_tanh", what="up")
    ref, S = oracle.linear_values_ref(oracle.dequantize_mx(*oracle.quantize_mx(f64(y2))), wh[2], f64(b[2]))
    assert_linear_close(y3, ref, S, what="down")


def test_empty_calls():
    d = dev()
    w = mx().mx_fp4_quantize_weight_slab(synth.make_weight(32, 64, seed=1).to(d))
    y = mx().mx_fp4_linear(torch.empty((0, 64), dtype=torch.bfloat16, device=d), w)
    assert y.shape == (0, 32)
    none = mx().FP4Slab(torch.empty((1, 0, 4, 16, 16), dtype=torch.uint8, device=d),
                        torch.empty((1, 0, 4), dtype=torch.uint8, device=d), 0, 64)
    assert mx().mx_fp4_linear(torch.zeros((3, 64), dtype=torch.bfloat16, device=d), none).shape == (3, 0)
