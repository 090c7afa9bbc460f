"""mx_fp4_experts at the ends of its ranges, on each of its kernels, and beside calls of
another shape in the same workspace."""

import pytest
import torch

from helpers import dev, mx
from test_gpu_experts import close, make, run

pytestmark = pytest.mark.gpu


# A few tokens; tiles of 128 weight rows; of 256.
@pytest.mark.parametrize("act", ["fp8", "fp4"])
@pytest.mark.parametrize("T,k,E,H,I", [(3, 1, 2, 65536, 32), (3, 2, 2, 32, 65536), (2, 64, 1024, 64, 32),
                                       (70, 1, 2, 65536, 32), (70, 1, 2, 32, 65536), (200, 1, 2, 65536, 32),
                                       (200, 1, 2, 32, 65536)])
def test_longest_rows_and_most_experts(T, k, E, H, I, act):
    print(f"experts T={T} k={k} E={E} H={H} I={I} {act}", flush=True)
    x, ids, w, up, down, uv, dv = make(T, k, E, H, I, seed=T)
    close(run(x, ids, w, up, down, act=act), x, ids, w, uv, dv, act)


def test_one_workspace_for_calls_of_every_kind_in_turn():
    # What a call leaves there (NaN codes and scales, a longer plan) reaches no later one.
    d = dev()
    made = [make(T, k, E, H, I, seed=T) for T, k, E, H, I in [(700, 2, 5, 544, 416), (9, 3, 5, 160, 96), (60, 2, 9, 288, 160),
                                                             (3000, 2, 6, 96, 64)]]
    need = max(mx().mx_fp4_experts_ws_bytes(x.shape[0], ids.shape[1], up.q.shape[0], x.shape[1], down.K, act)
               for x, ids, _, up, down, _, _ in made for act in ("fp8", "fp4"))
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device=d)
    want = {}
    for act in ("fp8", "fp4"):
        for i, (x, ids, w, up, down, uv, dv) in enumerate(made):
            want[act, i] = run(x, ids, w, up, down, act=act)
            close(want[act, i], x, ids, w, uv, dv, act)
    for order in ((0, 1, 2, 3), (3, 2, 1, 0), (1, 3, 0, 2)):
        for act in ("fp8", "fp4"):
            for i in order:
                x, ids, w, up, down, _, _ = made[i]
                nan = torch.full_like(x, float("nan"))
                run(nan, ids, w, up, down, act=act, workspace=ws)
                assert torch.equal(run(x, ids, w, up, down, act=act, workspace=ws), want[act, i]), (act, order, i)
