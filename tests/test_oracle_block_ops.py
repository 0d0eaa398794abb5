"""Pins of the float64 references in oracle/block_ops.py: hand-made selections, brute force, and
gradients against central differences."""
import numpy as np
import pytest

from oracle import block_ops as B
from oracle import moe_oracle as O


def test_groups_by_hand():
    # groups {0,1}, {2,3}, {4,5}; by maximum: 5, 4, 6; by the sum of two: 5, 8, 6.5
    l = np.array([[5.0, 0.0, 4.0, 4.0, 6.0, 0.5]])
    idx, _, _ = B.route_grouped(l, 2, 3, 1, "max", "softmax")
    assert idx.tolist() == [[4, 5]]
    idx, _, _ = B.route_grouped(l, 2, 3, 2, "max", "softmax")
    assert idx.tolist() == [[4, 0]]
    # sqrt(softplus) is close to sqrt(l): 2.24 + .83, 2 + 2, 2.45 + .99 -> the middle group
    idx, g, _ = B.route_grouped(l, 2, 3, 1, "top2", "sqrt_softplus")
    assert idx.tolist() == [[2, 3]] and np.allclose(g, 0.5)


def test_bias_selects_but_does_not_weigh_and_masks_win():
    l = np.array([[0.0, 0.0, 0.0, -np.inf]])
    idx, g, _ = B.route_grouped(l, 2, 1, 1, "max", "sigmoid", True, 1.0, np.array([0.0, 0.1, 0.2, 9.0]))
    assert idx.tolist() == [[2, 1]] and np.allclose(g, 0.5)
    idx, g, _ = B.route_grouped(np.full((1, 4), -np.inf), 3, 2, 2, "top2", "sigmoid", True, 1.0, np.ones(4))
    assert idx.tolist() == [[0, 1, 2]] and (g == 0).all()
    idx, g, _ = B.route_grouped(np.array([[np.nan, 1.0, -np.inf, np.inf]]), 3, 1, 1, "max", "softmax", False)
    assert idx.tolist() == [[3, 1, 0]] and g.tolist() == [[1.0, 0.0, 0.0]]


@pytest.mark.parametrize("score", ["softmax", "sigmoid", "sqrt_softplus"])
@pytest.mark.parametrize("renorm", [True, False])
def test_one_group_is_the_plain_routing(score, renorm):
    rng = np.random.default_rng(3)
    l = rng.standard_normal((20, 12))
    bias = rng.standard_normal(12) * 0.1
    for b in (None, bias):
        idx, g, _ = B.route_grouped(l, 4, 1, 1, "max", score, renorm, 1.5, b)
        want = O.top_k(O.selection_keys(l, score, b), 4)
        assert np.array_equal(idx, want)
        assert np.allclose(g, O.gates(l, want, score, renorm, 1.5), rtol=1e-12)


@pytest.mark.parametrize("score", ["softmax", "sigmoid", "sqrt_softplus"])
@pytest.mark.parametrize("renorm", [True, False])
def test_routing_gradient_against_differences(score, renorm):
    rng = np.random.default_rng(5)
    T, E, k = 3, 7, 3
    l = rng.standard_normal((T, E))
    idx = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    u, f = rng.standard_normal((T, k)), rng.random(E)
    args = (idx, u, score, renorm, 1.3, f, 0.7, 0.4)
    got = B.route_backward(l, *args)
    h = 1e-5
    for t in range(T):
        for e in range(E):
            a, b = l.copy(), l.copy()
            a[t, e] += h
            b[t, e] -= h
            d = (B.routing_loss(a, *args) - B.routing_loss(b, *args)) / (2 * h)
            # differences: h^2 / 6 times a third derivative below 50, and 1e-15 / h of rounding
            assert abs(d - got[t, e]) < 1e-8


def test_quantize_rows_by_hand():
    x = np.array([[1.0, -2.0, 0.5, 0.0], [0.0, 0.0, 0.0, 0.0], [np.inf, 1.0, 0.0, 0.0], [254.0, 1.0, 3.0, -5.0]],
                 np.float32)
    q, s = B.quantize_rows(x)
    assert q[0].tolist() == [64, -127, 32, 0] and s[0] == np.float32(2.0) / np.float32(127.0)
    assert (q[1] == 0).all() and s[1] == 0.0
    assert (q[2] == 0).all() and np.isnan(s[2])
    assert q[3].tolist() == [127, 0, 2, -2]                  # halves to even
    assert np.abs(q.astype(int)).max() <= 127


@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("pre", [False, True])
@pytest.mark.parametrize("G", [0, 1, 3, 6])
def test_block_norm_gradient_against_differences(post, pre, G):
    rng = np.random.default_rng(7)
    T, d, alpha, eps = 6, 4, 0.6, 1e-3
    v = dict(residual=rng.standard_normal((T, d)), y=rng.standard_normal((T, d)))
    v["post"] = rng.standard_normal(d) if post else None
    v["pre"] = rng.standard_normal(d) if pre else None
    v["gate"] = rng.standard_normal((G, d)) if G else None
    dx = rng.standard_normal((T, d))
    dn = rng.standard_normal((T, d)) if pre else None

    def loss(w):
        x, n = B.block_norm(w["residual"], w["y"], w["post"], w["gate"], alpha, w["pre"], eps)
        return (x * dx).sum() + (0.0 if n is None else (n * dn).sum())

    x, _ = B.block_norm(v["residual"], v["y"], v["post"], v["gate"], alpha, v["pre"], eps)
    got = B.block_norm_backward(dx, dn, x, v["y"], v["post"], v["gate"], alpha, v["pre"], eps)
    h = 1e-5
    for name, key in (("residual", "d_residual"), ("y", "d_y"), ("post", "d_post_weight"), ("gate", "d_gate"),
                      ("pre", "d_pre_weight")):
        if v[name] is None:
            assert got[key] is None
            continue
        for at in np.ndindex(v[name].shape):
            a, b = dict(v), dict(v)
            a[name], b[name] = v[name].copy(), v[name].copy()
            a[name][at] += h
            b[name][at] -= h
            d_ = (loss(a) - loss(b)) / (2 * h)
            # h^2 / 6 times a third derivative (below 1e4 for rows of four at this eps), and rounding
            assert abs(d_ - got[key][at]) < 1e-6


def test_combine_sum_skips_dropped_slots():
    rows = np.arange(12.0).reshape(4, 3)
    y = B.combine_sum(rows, np.array([[0, -1], [-1, -1], [3, 2]]), np.array([[2.0, 9.0], [1.0, 1.0], [1.0, 0.5]]),
                      np.ones((3, 3)))
    assert np.allclose(y, [2 * rows[0] + 1, np.ones(3), rows[3] + 0.5 * rows[2] + 1])
