"""Host checks of mx_fp4_linear_tile, which names the kernel of an MXFP4-weight
linear: its refusals, and that each kernel is some shape's."""

import ctypes

import pytest

from helpers import mx

INV, UNS = 1, 2


def test_refusals():
    L = mx().lib()
    a, b, c = ctypes.c_int(), ctypes.c_int(), ctypes.c_int()

    def call(M=8, K=128, N=32, act=1, out=(a, b, c)):
        return L.mx_fp4_linear_tile(M, K, N, act, *(None if o is None else ctypes.byref(o) for o in out))

    assert call() == 0
    for i in range(3):
        assert call(out=tuple(None if j == i else v for j, v in enumerate((a, b, c)))) == INV
    assert call(M=-1) == INV and call(K=40) == INV and call(N=-16) == INV and call(act=2) == INV
    assert call(act=0, K=96) == INV and call(N=24) == UNS and call(M=1 << 31) == UNS and call(N=1 << 21) == UNS
    assert call(M=1 << 30, N=1 << 20) == UNS
    a.value = b.value = c.value = 7
    assert call(M=0) == 0 and (a.value, b.value, c.value) == (0, 0, 0)
    with pytest.raises(ValueError):
        mx().mx_fp4_linear_tile(8, 128, 32, "fp6")
    with pytest.raises(mx().MXError):
        mx().mx_fp4_linear_tile(8, 128, 24)


def test_every_kernel_is_some_shapes():
    got = {act: set() for act in ("fp4", "fp8")}
    for act, seen in got.items():
        for M in [1, 16, 17, 300, *range(500, 9000, 250), 75348]:
            for N in (272, 2320, 5136, 7184, 8208, 15360):
                seen.add(mx().mx_fp4_linear_tile(M, 1024, N, act))
    few = (0, 0, False)
    assert got["fp4"] == {few, (128, 128, False), (256, 128, False), (256, 256, False), (256, 256, True)}
    assert got["fp8"] == {few, (128, 128, False), (192, 128, False), (256, 128, False), (256, 128, True)}


def test_a_call_without_workspace_is_the_few_token_kernels():
    for act in ("fp4", "fp8"):
        for M in (1, 7, 16):
            for N in (16, 4096, 15360):
                assert mx().mx_fp4_linear_ws_bytes(M, 5120, N, act) == 0
                assert mx().mx_fp4_linear_tile(M, 5120, N, act) == (0, 0, False)


def test_up_to_how_many_weight_rows_a_few_tokens_need_no_workspace():
    ws = mx().mx_fp4_linear_ws_bytes
    for K, rows in ((4096, 65536), (4128, 131072)):
        assert ws(16, K, rows, "fp4") == 0 and ws(16, K, rows + 16, "fp4") > 0
