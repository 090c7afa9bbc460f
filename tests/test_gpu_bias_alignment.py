"""A bias at any 2-byte aligned address, as a slice of a flat parameter buffer
has: each kernel gives the bits that it gives with a 256-byte aligned copy.
N is no multiple of any tile, so that the last weight rows' bias ends inside
one; what follows it in the buffer is NaN."""

import pytest
import torch

import synth
from helpers import dev, mx

pytestmark = pytest.mark.gpu


def same(a, b):
    return torch.equal(a.view(torch.int16), b.view(torch.int16))


def biases(N, seed):
    """An aligned bias, and the same values 2, 4 and 6 bytes past an aligned address."""
    g = torch.Generator().manual_seed(seed)
    b = (8 * torch.randn((N,), generator=g)).to(torch.float16).to(dev())
    assert b.data_ptr() % 16 == 0
    shifted = []
    for off in (1, 2, 3):
        buf = torch.full((N + 8,), float("nan"), dtype=torch.float16, device=dev())
        v = buf[off : off + N]
        v.copy_(b)
        assert v.data_ptr() % 8 == 2 * off
        shifted.append(v)
    return b, shifted


FEW = (0, 0, False)


@pytest.mark.parametrize("act,M,N,tile", [
    ("fp4", 3, 272, FEW), ("fp4", 90, 528, FEW), ("fp4", 385, 2320, (128, 128, False)),
    ("fp4", 903, 4112, (256, 128, False)), ("fp4", 1051, 7184, (256, 256, False)), ("fp4", 2198, 7184, (256, 256, True)),
    ("fp8", 3, 272, FEW), ("fp8", 90, 528, FEW), ("fp8", 385, 2320, (128, 128, False)),
    ("fp8", 903, 4112, (192, 128, False)), ("fp8", 644, 8208, (256, 128, False)), ("fp8", 1051, 7184, (256, 128, True)),
])
def test_mxfp4_linears(act, M, N, tile):
    print(f"bias alignment fp4 M={M} N={N} {act}", flush=True)
    K = 320
    assert mx().mx_fp4_linear_tile(M, K, N, act) == tile
    x = synth.make_activation(M, K, seed=M).to(dev())
    w = mx().mx_fp4_quantize_weight_slab(synth.make_weight(N, K, seed=N).to(dev()))
    b, shifted = biases(N, M + N)
    y = mx().mx_fp4_linear(x, w, b, act=act)
    plain = mx().mx_fp4_linear(x, w, None, act=act)
    # The bias is in every column: it is large against the products here.
    assert bool(((y - plain).float() - b.float()).abs().max() < 0.5)
    for v in shifted:
        assert same(mx().mx_fp4_linear(x, w, v, act=act), y)


@pytest.mark.parametrize("M,N", [(300, 272), (520, 784)])
@pytest.mark.parametrize("kind", ["slab", "m128", "splitk", "small", "small split", "balanced", "requant", "per channel",
                                  "row-major", "row-major, K % 128 = 64", "fused", "one call"])
def test_mxfp8_linears(kind, M, N):
    print(f"bias alignment {kind} M={M} N={N}", flush=True)
    m = mx()
    K = 320 if kind == "row-major, K % 128 = 64" else 512
    if kind == "requant":
        N = N // 64 * 64
    x = synth.make_activation(M, K, seed=M).to(dev())
    w = synth.make_weight(N, K, seed=N).to(dev())
    xs, ws = m.mx_quantize_act_slab(x), m.mx_quantize_weight_slab(w)
    xr, wr = m.mx_quantize_act(x), m.mx_quantize_weight(w)
    xp, wp = m.mx_pc_quantize_act_slab(x), m.mx_pc_quantize_weight_slab(w)

    def run(b):
        if kind == "requant":
            out = m.mx_linear_slab_requant(xs, ws, b)
            return torch.cat([out.q.reshape(-1), out.s.reshape(-1)])
        y = {
            "slab": lambda: m.mx_linear_slab(xs, ws, b),
            "m128": lambda: m.mx_linear_slab_m128(xs, ws, b),
            "splitk": lambda: m.mx_linear_slab_splitk(xs, ws, b, splits=2),
            "small": lambda: m.mx_linear_slab_small(xs, ws, b, splits=1),
            "small split": lambda: m.mx_linear_slab_small(xs, ws, b, splits=2),
            "balanced": lambda: m.mx_linear_slab_balanced(xs, ws, b),
            "per channel": lambda: m.mx_pc_linear_slab(xp, wp, b),
            "fused": lambda: m.mx_linear_fused(x, *wr, b),
            "one call": lambda: m.mx_linear(x, ws, b),
        }.get(kind, lambda: m.mx_linear_q(*xr, *wr, b))()
        return y.view(torch.int16)

    b, shifted = biases(N, M + N)
    y = run(b)
    assert not torch.equal(y, run(None))
    for v in shifted:
        assert torch.equal(run(v), y)
