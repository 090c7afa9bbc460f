"""Each kernel of the MXFP4-weight linears, the tiled ones above all, under
what a serving program does to it: non-finite groups, calls behind other calls,
captured graphs, two streams at once. Every case states the kernel that it is
for and asks the library that it is the one.

K of 352 and 320 end inside a 128-K slab (96 and 64 of it), so what the kernels
read past K counts in every case."""

import numpy as np
import pytest
import torch

import oracle
import synth
from helpers import assert_linear_close, dev, f64, mx
from test_gpu_fp4_limits import last_rows, random_fp4, random_fp8, same

pytestmark = pytest.mark.gpu

FEW = (0, 0, False)
TILES = [
    ("fp4", 385, 2320, (128, 128, False)), ("fp4", 903, 4112, (256, 128, False)), ("fp4", 1051, 7184, (256, 256, False)),
    ("fp4", 2198, 7184, (256, 256, True)),
    ("fp8", 385, 2320, (128, 128, False)), ("fp8", 903, 4112, (192, 128, False)), ("fp8", 644, 8208, (256, 128, False)),
    ("fp8", 1051, 7184, (256, 128, True)),
]
KERNELS = [("fp4", 3, 272, FEW), ("fp4", 90, 528, FEW), ("fp8", 3, 272, FEW), ("fp8", 90, 528, FEW)] + TILES


def case(act, M, N, tile, K=None):
    K = K or (352 if act == "fp4" else 320)
    print(f"fp4 kernel {tile} {act} {M}x{K}x{N}", flush=True)
    assert mx().mx_fp4_linear_tile(M, K, N, act) == tile
    return K


def quantized(x, act):
    return mx().mx_fp4_quantize_act_slab(x) if act == "fp4" else mx().mx_quantize_act_slab(x)


def weights(N, K, seed):
    return mx().mx_fp4_quantize_weight_slab(synth.make_weight(N, K, seed=seed).to(dev()))


@pytest.mark.parametrize("act,M,N,tile", KERNELS)
def test_nonfinite_groups(act, M, N, tile):
    """A NaN or Inf in a token's group makes that token's outputs NaN, one in a
    weight row's group that column's; nothing else changes. In the first slab, in
    the middle and in the last group of the partial slab."""
    K = case(act, M, N, tile)
    d = dev()
    x = synth.make_activation(M, K, seed=2)
    w = synth.make_weight(N, K, seed=3)
    clean = mx().mx_fp4_linear(x.to(d), mx().mx_fp4_quantize_weight_slab(w.to(d)), act=act)
    assert bool(torch.isfinite(clean).all())
    rows, cols = [1, M // 2, M - 1], [5, N // 2, N - 1]
    for r, k, v in zip(rows, (K - 1, 0, 200), ("inf", "nan", "-inf")):
        x[r, k] = float(v)
    for c, k, v in zip(cols, (0, K - 1, 140), ("nan", "-inf", "nan")):
        w[c, k] = float(v)
    y = mx().mx_fp4_linear(x.to(d), mx().mx_fp4_quantize_weight_slab(w.to(d)), act=act)
    want = torch.zeros((M, N), dtype=torch.bool)
    want[rows] = True
    want[:, cols] = True
    assert torch.equal(torch.isnan(y).cpu(), want)
    keep = (~want).to(d)
    assert torch.equal(y[keep], clean[keep])


@pytest.mark.parametrize("act,M,N,tile", KERNELS)
def test_a_nan_scale_marks_its_group_whatever_the_codes(act, M, N, tile):
    """Operands quantized elsewhere: scale 0xFF over zero codes, as
    mx_fp4_dequantize_slab reads it."""
    K = case(act, M, N, tile)
    x = quantized(synth.make_activation(M, K, seed=4).to(dev()), act)
    w = weights(N, K, 5)
    y = mx().mx_fp4_linear_slab(x, w)
    r, c = M - 2, N - 3
    if act == "fp4":
        x.q[K // 128, r // 16, (K % 128) // 32 - 1, r % 16] = 0
        x.s[K // 128, r, (K % 128) // 32 - 1] = 0xFF
    else:
        x.q[K // 64 - 1, r, 32:] = 0
        x.s[K // 64 - 1, r, 1] = 0xFF
    w.q[0, c // 16, 1, c % 16] = 0
    w.s[0, c, 1] = 0xFF
    z = mx().mx_fp4_linear_slab(x, w)
    want = torch.zeros((M, N), dtype=torch.bool, device=dev())
    want[r] = True
    want[:, c] = True
    assert torch.equal(torch.isnan(z), want)
    assert torch.equal(z[~want], y[~want])


@pytest.mark.parametrize("K", [32, 96, 352])
@pytest.mark.parametrize("act,M,N,tile", KERNELS)
def test_nothing_is_left_from_the_call_before(act, M, N, tile, K):
    """Fewer steps than a ring holds, behind a call whose operands are NaN
    throughout: stale codes or scales would be NaN here."""
    K = case(act, M, N, tile, K if act == "fp4" else (K + 63) // 64 * 64)
    d = dev()
    x, w = synth.make_activation(M, K, seed=6).to(d), weights(N, K, 7)
    y = mx().mx_fp4_linear(x, w, act=act)
    nan = torch.full((max(M, N), 1536), float("nan"), dtype=torch.bfloat16, device=d)
    wn = mx().mx_fp4_quantize_weight_slab(nan[:N])
    assert bool(torch.isnan(mx().mx_fp4_linear(nan[:M], wn, act=act)).all())
    z = mx().mx_fp4_linear(x, w, act=act)
    assert bool(torch.isfinite(z).all()) and same(z, y)


@pytest.mark.parametrize("act,M,N,tile", KERNELS)
def test_rows_are_independent_of_their_batch(act, M, N, tile):
    K = case(act, M, N, tile)
    x = synth.make_activation(M, K, seed=8).to(dev())
    w = weights(N, K, 9)
    y = mx().mx_fp4_linear(x, w, act=act)
    z = x.clone()
    z[M // 2 :] = float("nan")
    yz = mx().mx_fp4_linear(z, w, act=act)
    assert same(yz[: M // 2], y[: M // 2])
    assert bool(torch.isnan(yz[M // 2 :]).all())


@pytest.mark.parametrize("act,M,N,tile", KERNELS)
def test_graph_replays_match_eager(act, M, N, tile):
    """Two graphs, each with a workspace of its own, replayed in turn."""
    K = case(act, M, N, tile)
    d = dev()
    w = weights(N, K, 10)
    b = synth.make_bias(N, seed=1).to(d)
    ins = [synth.make_activation(M, K, seed=s).to(d) for s in (1, 2, 3)]
    want = [mx().mx_fp4_linear(x, w, b, gelu=True, act=act) for x in ins]
    graphs = []
    for k in range(2):
        x = ins[k].clone()
        y = torch.empty((M, N), dtype=torch.bfloat16, device=d)
        ws = torch.empty((max(mx().mx_fp4_linear_ws_bytes(M, K, N, act), 1),), dtype=torch.uint8, device=d)

        def step():
            mx().mx_fp4_linear(x, w, b, gelu=True, act=act, y=y, workspace=ws)

        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append((g, x, y, ws))
    for turn in range(6):
        g, x, y, ws = graphs[turn % 2]
        k = (2 * turn + 1) % 3
        x.copy_(ins[k])
        y.fill_(7)
        ws.fill_(0xFF)
        g.replay()
        mx().mx_fp4_linear(ins[turn % 3], w, act=act)  # eager work between replays
        torch.cuda.synchronize()
        assert same(y, want[k]), turn
    del graphs


@pytest.mark.parametrize("act,M,N,tile", KERNELS)
def test_two_streams_at_once(act, M, N, tile):
    K = case(act, M, N, tile)
    d = dev()
    w = weights(N, K, 11)
    xs = [synth.make_activation(M, K, seed=s).to(d) for s in (4, 5)]
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


@pytest.mark.parametrize("act,K", [("fp4", 8224), ("fp8", 8256)])
@pytest.mark.parametrize("M", [17, 33, 250])
def test_long_rows_of_more_than_16_tokens(M, act, K):
    """16 x 16 tiles on long rows: sixteen waves."""
    N = 272
    case(act, M, N, FEW, K)
    x, w, b = synth.make_activation(M, K, seed=M), synth.make_weight(N, K, seed=N) * 4, synth.make_bias(N, seed=K)
    d = dev()
    y = mx().mx_fp4_linear(x.to(d), mx().mx_fp4_quantize_weight_slab(w.to(d)), b.to(d), gelu=True, act=act)
    xh = oracle.dequantize_fp4(*oracle.quantize_fp4(f64(x))) if act == "fp4" else oracle.dequantize_mx(
        *oracle.quantize_mx(f64(x)))
    ref, S = oracle.linear_values_ref(xh, oracle.dequantize_fp4(*oracle.quantize_fp4(f64(w))), f64(b), "gelu_tanh")
    assert_linear_close(y, ref, S, "gelu_tanh", what=f"{M}x{K}x{N} {act}")


@pytest.mark.parametrize("act", ["fp4", "fp8"])
def test_halved_tiles_past_4_gib(act):
    """The last rows are those of a call on them alone, the halved last round's
    among them."""
    M, K, N = 139_300, 128, 16_384
    case(act, M, N, (256, 256, True) if act == "fp4" else (256, 128, True), K)
    assert M * N * 2 > 1 << 32
    x = (random_fp4 if act == "fp4" else random_fp8)(M, K, 1)
    w = random_fp4(N, K, 2)
    y = mx().mx_fp4_linear_slab(x, w)
    t = last_rows(x, 1024)
    assert mx().mx_fp4_linear_tile(t.rows, K, N, act) != FEW  # tiles too: the same chain of products
    assert same(y[-t.rows :], mx().mx_fp4_linear_slab(t, w))


def to_slab(codes, scales, act):
    d = dev()
    if act == "fp4":
        q, s = oracle.fp4_slab(codes, scales)
        return mx().FP4Slab(torch.from_numpy(q).to(d), torch.from_numpy(s).to(d), *codes.shape)
    M, K = codes.shape
    R = (M + 255) // 256 * 256
    q, s = np.zeros((K // 64, R, 64), np.uint8), np.zeros((K // 64, R, 2), np.uint8)
    q[:, :M] = codes.reshape(M, -1, 64).transpose(1, 0, 2)
    s[:, :M] = scales.reshape(M, -1, 2).transpose(1, 0, 2)
    return mx().Slab(torch.from_numpy(q).to(d), torch.from_numpy(s).to(d), M)


@pytest.mark.parametrize("act,M,N,tile", KERNELS)
def test_sums_that_fp32_holds_are_exact(act, M, N, tile):
    """Operands whose partial sums all fit in 24 bits, in whatever order they are
    added: the outputs are the exact sums rounded once, bit for bit, so that one
    product lost, doubled or scaled by a neighbour's scale shows.

    Group g has a scale of 2^d on the tokens and 2^-d on the weights, d from -127
    to 127, each times 1/2, 1 or 2 by row: every scale code but NaN, and products'
    scales from 1/4 to 4. E2M1 values are multiples of 1/2 up to 6; E4M3 ones are
    kept to magnitudes 1 to 1.875, multiples of 1/8. A product is then a multiple
    of u = 2^-4 (E4M3: 2^-6) of at most 36 x 4 = 2304 u (11.25 x 4 = 2880 u), and
    with K <= 1088 and a bias that is a whole number up to 64 (4096 u), every
    partial sum is below 1088 x 2880 + 4096 < 2^22 u."""
    K = case(act, M, N, tile, 1088 if M < 200 else 352 if act == "fp4" else 320)
    rng = np.random.default_rng(M + N)
    G = K // 32
    d = rng.integers(-127, 128, G)
    d[: min(G, 2)] = [-127, 127][: min(G, 2)]
    sx = np.clip(127 + d + rng.integers(-1, 2, (M, G)), 0, 254).astype(np.uint8)
    sw = np.clip(127 - d + rng.integers(-1, 2, (N, G)), 0, 254).astype(np.uint8)
    wc = rng.integers(0, 16, (N, K)).astype(np.uint8)
    if act == "fp4":
        xc = rng.integers(0, 16, (M, K)).astype(np.uint8)
        xh = oracle.dequantize_fp4(xc, sx)
    else:
        xc = (0x38 + rng.integers(0, 8, (M, K)) + 128 * rng.integers(0, 2, (M, K))).astype(np.uint8)
        xh = oracle.dequantize_mx(xc, sx)
    b = rng.integers(-64, 65, N).astype(np.float64)
    exact = xh @ oracle.dequantize_fp4(wc, sw).T + b  # exact in float64 too
    y = mx().mx_fp4_linear_slab(to_slab(xc, sx, act), to_slab(wc, sw, "fp4"), torch.from_numpy(b).half().to(dev()))
    assert np.array_equal(f64(y), oracle.bf16_round(exact))


@pytest.mark.parametrize("act,tiles", [
    ("fp4", {300: (128, 128, False), 800: (256, 128, False), 1600: (256, 256, False), 3100: (256, 256, True)}),
    ("fp8", {300: (128, 128, False), 800: (192, 128, False), 1200: (256, 128, False), 1600: (256, 128, True)}),
])
def test_every_tile_adds_in_the_same_order(act, tiles):
    """A token's outputs are the same bits on tiles of every shape. The second half
    of K holds the first's groups in another order with the weights negated, over
    many binades, so that what is left is the sums' rounding, which shows their
    order."""
    K, N = 2048, 5136
    d = dev()
    g = torch.Generator(device=d).manual_seed(12)
    n, M = K // 64, max(tiles)
    x = torch.randn((M, n, 32), generator=g, device=d) * torch.exp2(8 * torch.randn((1, n, 1), generator=g, device=d))
    w = torch.randn((N, n, 32), generator=g, device=d)
    order = torch.randperm(n, generator=g, device=d)
    x = torch.cat([x, x[:, order]], 1).reshape(M, K).to(torch.bfloat16)
    ws = mx().mx_fp4_quantize_weight_slab(torch.cat([w, -w[:, order]], 1).reshape(N, K))
    ys = {}
    for m, tile in tiles.items():
        case(act, m, N, tile, K)
        ys[m] = mx().mx_fp4_linear(x[:m], ws, act=act)
    first = min(tiles)
    assert bool((ys[first] != 0).any())
    for m, y in ys.items():
        assert same(y[:first], ys[first]), tiles[m]
    # The few-token kernel's order is another one, which these inputs show.
    few = mx().mx_fp4_linear(x[:100], ws, act=act)
    case(act, 100, N, FEW, K)
    assert not same(few, ys[first][:100])
