"""Row-major scales are bytes and may start at any address: the row-major
linear on pre-quantized operands whose scales are slices of larger buffers."""

import pytest
import torch

import oracle
import synth
from helpers import assert_linear_close, dev, f64, mx, quant_ref

pytestmark = pytest.mark.gpu


def at(s, off):
    buf = torch.full((s.numel() + 8,), 0xFF, dtype=torch.uint8, device=s.device)
    v = buf[off : off + s.numel()].view(s.shape)
    v.copy_(s)
    assert v.data_ptr() % 4 == off % 4
    return v


@pytest.mark.parametrize("off", [(1, 0), (0, 2), (3, 3), (4, 4)])
@pytest.mark.parametrize("K", [256, 320])
def test_row_major_linear(K, off):
    M, N = 300, 272
    print(f"scale alignment K={K} {off}", flush=True)
    d = dev()
    x, w, b = synth.make_activation(M, K, 1), synth.make_weight(N, K, 2), synth.make_bias(N, 3)
    xq, xs = mx().mx_quantize_act(x.to(d))
    wq, ws = mx().mx_quantize_weight(w.to(d))
    y = mx().mx_linear_q(xq, at(xs, off[0]), wq, at(ws, off[1]), b.to(d), gelu=True)
    yref, S = oracle.linear_ref(*quant_ref(x), *quant_ref(w), bias=f64(b), epilogue="gelu_tanh")
    assert_linear_close(y, yref, S, "gelu_tanh", what=f"K={K} {off}")
