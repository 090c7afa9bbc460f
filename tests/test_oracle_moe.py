"""The references of routing, experts and block norms against small cases worked
out by hand or by another route."""

import numpy as np
import pytest

import oracle

INF, NAN = np.inf, np.nan


def test_route_takes_the_highest_and_ties_go_to_the_lower_index():
    ids, w = oracle.route_ref([[1.0, 3.0, 3.0, 2.0]], 3, renorm=False)
    p = np.exp([1.0, 3.0, 3.0, 2.0])
    assert ids.tolist() == [[1, 2, 3]]
    assert np.allclose(w[0], (p / p.sum())[[1, 2, 3]], rtol=1e-15)


def test_route_masks():
    ids, w = oracle.route_ref([[-INF, 5.0, NAN, INF], [-INF] * 4], 3)
    assert ids.tolist() == [[3, 1, 0], [0, 1, 2]]  # the masked ones last, lowest first
    assert w[0].tolist() == [1.0, 0.0, 0.0]  # exp(5 - f32 max) is 0
    assert w[1].tolist() == [0.0, 0.0, 0.0]


def test_route_bias_steers_the_choice_only():
    ids, w = oracle.route_ref([[0.0, 1.0, 2.0]], 1, scores="sigmoid", bias=[5.0, 0.0, 0.0], renorm=False, scale=2.0)
    assert ids.tolist() == [[0]] and w[0, 0] == 1.0  # 2 sigmoid(0)


def test_route_groups():
    # Highest logit in group 1; by the sum of two with a bias, group 0 wins.
    l = [[2.0, 1.9, 2.1, -9.0]]
    assert oracle.route_ref(l, 2, groups=2)[0].tolist() == [[2, 3]]
    assert oracle.route_ref(l, 2, scores="sigmoid", bias=[0.0] * 4, groups=2)[0].tolist() == [[0, 1]]


@pytest.mark.parametrize("act", ["fp4", "fp8"])
def test_experts_reduce_to_one_dense_block(act):
    rng = np.random.default_rng(3)
    T, H, I = 5, 64, 32
    x = oracle.bf16_round(rng.standard_normal((T, H)))
    up, down = rng.standard_normal((1, 2 * I, H)), rng.standard_normal((1, H, I))
    y, tol = oracle.experts_ref(x, np.zeros((T, 1), int), np.full((T, 1), 0.5), up, down, act, "silu")
    xh = oracle.activation_values(x, act)
    g, u = xh @ up[0, :I].T, xh @ up[0, I:].T
    a = oracle.bf16_round(g / (1 + np.exp(-g)) * u)
    assert np.allclose(y, 0.5 * oracle.activation_values(a, act) @ down[0].T, rtol=1e-12)
    assert (tol > 0).all()


def test_experts_skip_and_repeat():
    rng = np.random.default_rng(4)
    x = oracle.bf16_round(rng.standard_normal((2, 32)))
    up, down = rng.standard_normal((2, 64, 32)), rng.standard_normal((2, 32, 32))
    one, _ = oracle.experts_ref(x, np.array([[0, -1], [7, -3]]), np.ones((2, 2)), up, down, "fp8", "gelu")
    two, _ = oracle.experts_ref(x, np.array([[0, 0], [1, 0]]), np.array([[0.25, 0.75], [0.0, 0.0]]), up, down, "fp8", "gelu")
    assert np.allclose(one[0], two[0], rtol=1e-12) and not one[1].any() and not two[1].any()


def test_block_norm_is_the_rms_norm_without_its_options():
    rng = np.random.default_rng(5)
    x, r = oracle.bf16_round(rng.standard_normal((3, 64))), oracle.bf16_round(rng.standard_normal((3, 64)))
    w = oracle.bf16_round(rng.standard_normal(64))
    h, y = oracle.rmsnorm_ref(x, r, w)
    hv, _ = oracle.block_h_ref(x, r)
    assert np.array_equal(oracle.bf16_round(hv), h)
    yv, err = oracle.block_y_ref(h, weight=w)
    assert np.array_equal(oracle.bf16_round(yv), y) and (err >= 0).all()


def test_block_norm_layer_and_modulation():
    h = np.array([[1.0, 2.0, 3.0, 6.0]])
    y, _ = oracle.block_y_ref(h, kind="layer", scale=np.full(4, 1.0), shift=np.full(4, 3.0), eps=0.0)
    assert np.allclose(y, (h - 3.0) / np.sqrt(3.5) * 2.0 + 3.0, rtol=1e-15)
