"""GPU parity of the MXFP4 quantizers, the dequantizer and the layout
conversions against the oracle: codes, scales and values bit for bit. The
rule is exact on every finite bf16 and f32 input, so nothing here has a
tolerance."""

import numpy as np
import pytest
import torch

import oracle
import synth
from helpers import dev, f64, mx, u8

pytestmark = pytest.mark.gpu


def check_slab(slab, x, what=""):
    q, s = oracle.fp4_slab(*oracle.quantize_fp4(f64(x)))
    assert np.array_equal(u8(slab.s), s), f"{what}: scales"
    assert np.array_equal(u8(slab.q), q), f"{what}: codes"


@pytest.mark.parametrize("M,K", [(1, 32), (1, 5120), (15, 96), (16, 128), (77, 160), (256, 512), (257, 544), (300, 672),
                                 (513, 64), (40, 13824)])
def test_act_quantizer_matches_oracle(M, K):
    print(f"fp4 act M={M} K={K}", flush=True)
    x = synth.make_activation(M, K, seed=M + K)
    check_slab(mx().mx_fp4_quantize_act_slab(x.to(dev())), x, f"{M}x{K}")


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("N,K", [(1, 32), (100, 96), (272, 1056)])
def test_weight_quantizer_matches_oracle(N, K, dtype):
    print(f"fp4 weight N={N} K={K} {dtype}", flush=True)
    w = synth.make_weight(N, K, seed=N).to(dtype)
    check_slab(mx().mx_fp4_quantize_weight_slab(w.to(dev())), w, f"{N}x{K}")


def test_every_bf16_value_under_many_scales():
    """Each of the 65536 bf16 patterns, in groups led by a power of two that
    sets the shared exponent at, just above or far above the value's own."""
    print("fp4 exhaustive bf16", flush=True)
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    vals = bits.view(torch.bfloat16)
    rows = []
    for lead in (None, 2.0**-126, 2.0**-20, 1.0, 4.0, 2.0**100):
        g = vals[: 65536 // 31 * 31].view(-1, 31)
        first = torch.zeros(g.shape[0], 1, dtype=torch.bfloat16) if lead is None else torch.full(
            (g.shape[0], 1), lead, dtype=torch.bfloat16)
        rows.append(torch.cat([first, g], dim=1))
    rows.append(vals.view(-1, 32)[-1:].clone())
    x = torch.cat(rows)
    check_slab(mx().mx_fp4_quantize_act_slab(x.to(dev())), x)


def test_f32_ties_subnormals_and_special_rows():
    print("fp4 f32 specials", flush=True)
    rng = np.random.default_rng(3)
    w = np.zeros((12, 64), dtype=np.float32)
    mids = np.array([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=np.float32)
    near = np.concatenate([mids, np.nextafter(mids, np.float32(9)), np.nextafter(mids, np.float32(0)), -mids])
    w[0, : near.size] = near
    w[0, 31] = w[0, 63] = 4.0
    w[1] = w[0] * np.float32(2.0**-129)  # subnormal amax: the clamped exponent
    w[2] = rng.standard_normal(64).astype(np.float32) * np.float32(2.0**120)
    w[2, 5] = np.finfo(np.float32).max
    w[3, 7] = np.nan
    w[4, 40] = np.inf
    w[5, 3] = -np.inf
    w[6] = -0.0
    w[7] = np.float32(2.0**-149)
    w[8] = rng.integers(0, 2**32, 64, dtype=np.uint32).view(np.float32)
    w[9] = 7.9999995  # saturates at 6 times the scale
    w[10, ::2] = -1e-30
    w[11] = near.max() * rng.standard_normal(64)
    x = torch.from_numpy(w)
    check_slab(mx().mx_fp4_quantize_weight_slab(x.to(dev())), x)


def test_strided_rows_and_reused_output():
    print("fp4 strided", flush=True)
    d = dev()
    base = synth.make_activation(300, 512, seed=5).to(d)
    x = base[:, 64:416]  # K = 352, pitch 512
    out = mx().mx_fp4_quantize_act_slab(x.contiguous())
    out.q.fill_(0xA5)
    out.s.fill_(0xA5)
    got = mx().mx_fp4_quantize_act_slab(x, out=out)
    assert got is out
    check_slab(out, x)  # pad rows and groups are zeroed again


def random_fp4(rows, K, seed, scales=None):
    rng = np.random.default_rng(seed)
    c = rng.integers(0, 16, (rows, K)).astype(np.uint8)
    s = (rng.integers(0, 256, (rows, K // 32)) if scales is None else scales).astype(np.uint8)
    return c, s


def to_slab(c, s):
    q, sc = oracle.fp4_slab(c, s)
    d = dev()
    return mx().FP4Slab(torch.from_numpy(q).to(d), torch.from_numpy(sc).to(d), c.shape[0], c.shape[1])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,K", [(1, 32), (64, 256), (273, 736)])
def test_dequantize_every_scale(rows, K, dtype):
    print(f"fp4 dequantize {rows}x{K} {dtype}", flush=True)
    c, s = random_fp4(rows, K, rows)
    if s.size >= 512:
        s.reshape(-1)[:512] = np.tile(np.arange(256), 2)
    with np.errstate(over="ignore"):
        want = torch.from_numpy(oracle.dequantize_fp4(c, s)).float().to(dtype)
    got = mx().mx_fp4_dequantize_slab(to_slab(c, s), dtype=dtype).cpu()
    nan = torch.isnan(want)
    assert torch.equal(torch.isnan(got), nan)
    assert torch.equal(got[~nan], want[~nan])
    assert torch.equal(torch.signbit(got[~nan]), torch.signbit(want[~nan]))


def test_dequantize_into_strided_rows_leaves_the_rest():
    print("fp4 dequantize strided", flush=True)
    c, s = random_fp4(37, 160, 1, np.full((37, 5), 120))
    big = torch.full((40, 192), 7.0, dtype=torch.bfloat16, device=dev())
    mx().mx_fp4_dequantize_slab(to_slab(c, s), y=big[1:38, 16:176])
    want = torch.full((40, 192), 7.0, dtype=torch.bfloat16)
    want[1:38, 16:176] = torch.from_numpy(oracle.dequantize_fp4(c, s)).to(torch.bfloat16)
    assert torch.equal(big.cpu(), want)


@pytest.mark.parametrize("rows,K", [(1, 32), (19, 160), (256, 128), (300, 1056)])
def test_pack_row_major(rows, K):
    print(f"fp4 pack {rows}x{K}", flush=True)
    c, s = random_fp4(rows, K, K)
    d = dev()
    slab = mx().mx_fp4_slab_pack(torch.from_numpy(oracle.pack_rows(c)).to(d), torch.from_numpy(s).to(d))
    q, sc = oracle.fp4_slab(c, s)
    assert np.array_equal(u8(slab.q), q) and np.array_equal(u8(slab.s), sc)


@pytest.mark.parametrize("rows,K", [(1, 64), (19, 192), (256, 128), (300, 1088)])
def test_unpack_to_mxfp8_keeps_every_value(rows, K):
    print(f"fp4 unpack {rows}x{K}", flush=True)
    c, s = random_fp4(rows, K, K + 1)
    slab = mx().mx_fp4_slab_unpack(to_slab(c, s))
    R = slab.q.shape[1]
    q = u8(slab.q)
    assert not q[:, rows:].any() and not u8(slab.s)[:, rows:].any()
    q = q[:, :rows].transpose(1, 0, 2).reshape(rows, K)
    s8 = u8(slab.s)[:, :rows].transpose(1, 0, 2).reshape(rows, K // 32)
    assert R == (rows + 255) // 256 * 256
    assert np.array_equal(s8, s)
    a, b = oracle.dequantize_mx(q, s8), oracle.dequantize_fp4(c, s)
    assert np.array_equal(a, b, equal_nan=True)
    assert np.array_equal(np.signbit(a), np.signbit(b))
    assert (q.reshape(rows, -1, 32)[s == 255] == 0x7F).all()


def test_offsets_past_32_bits():
    """An operand of more than 2^32 elements: rows at its end, against the
    quantizer on those rows alone."""
    print("fp4 large", flush=True)
    d = dev()
    M, K = 300_032, 14_336  # 4.3e9 elements, 8.6 GB of bf16
    x = torch.empty((M, K), dtype=torch.bfloat16, device=d)
    x.fill_(0.5)
    tail = synth.make_activation(272, K, seed=6).to(d)
    x[-272:] = tail
    slab = mx().mx_fp4_quantize_act_slab(x)
    del x
    ref = mx().mx_fp4_quantize_act_slab(tail)
    blk = (M - 272) // 16
    assert (M - 272) % 16 == 0
    assert torch.equal(slab.q[:, blk : blk + 17], ref.q[:, :17])
    assert torch.equal(slab.s[:, M - 272 : M], ref.s[:, :272])
    assert not bool(slab.s[:, M:].any())
    y = mx().mx_fp4_dequantize_slab(slab)
    assert torch.equal(y[-272:], mx().mx_fp4_dequantize_slab(ref))
    assert bool((y[1000] == 0.5).all())


def test_empty_operands():
    d = dev()
    x = torch.empty((0, 64), dtype=torch.bfloat16, device=d)
    slab = mx().mx_fp4_quantize_act_slab(x)
    assert slab.q.numel() == 0
    assert mx().mx_fp4_dequantize_slab(slab).shape == (0, 64)
    assert mx().mx_fp4_slab_unpack(slab).q.numel() == 0
