"""Pins of the gated linear recurrence's and the q / k norm-with-rotation
oracles: closed forms and finite differences, none through the code they pin."""

import numpy as np
import pytest

from oracle import (gated_delta_rule_forward, linear_backward, linear_forward, norm_rope,
                    norm_rope_backward, rotate, rotation_angles)


def _draw(rng, B=1, H=2, Hqk=2, L=6, dk=4, dv=3):
    q, k = rng.standard_normal((2, B, Hqk, L, dk))
    v = rng.standard_normal((B, H, L, dv))
    g = -rng.exponential(0.5, (B, H, L))
    return q, k, v, g, rng.standard_normal((B, H, dk, dv))


def test_forward_is_the_masked_product_with_decay():
    q, k, v, g, S0 = _draw(np.random.default_rng(0))
    o, S = linear_forward(q, k, v, g, S0)
    G = np.cumsum(g, -1)
    want = np.exp(G)[..., None] * (q @ S0)
    for r in range(6):
        for i in range(r + 1):
            f = np.exp(G[..., r] - G[..., i]) * (q[:, :, r] * k[:, :, i]).sum(-1)
            want[:, :, r] += f[..., None] * v[:, :, i]
    np.testing.assert_allclose(o, want, rtol=1e-12, atol=1e-13)
    last = np.exp(G[..., -1])[..., None, None] * S0
    for i in range(6):
        last = last + np.exp(G[..., -1] - G[..., i])[..., None, None] \
            * k[:, :, i, :, None] * v[:, :, i, None, :]
    np.testing.assert_allclose(S, last, rtol=1e-12, atol=1e-13)


def test_orthonormal_keys_make_it_the_gated_delta_rule():
    """With orthonormal keys and a zero state the delta reads nothing, so the
    (separately pinned) gated delta rule with beta = 1 writes the same."""
    rng = np.random.default_rng(1)
    q, _, v, g, _ = _draw(rng, L=4)
    k = np.broadcast_to(np.linalg.qr(rng.standard_normal((4, 4)))[0], q.shape)
    a = gated_delta_rule_forward(q, k, v, np.exp(g), np.ones(g.shape))
    b = linear_forward(q, k, v, g)
    for x, y in zip(a, b):
        np.testing.assert_allclose(x, y, rtol=1e-12, atol=1e-13)


def test_wipe_separates_documents():
    q, k, v, g, S0 = _draw(np.random.default_rng(2), L=7)
    g[..., 3] = -np.inf
    o, S = linear_forward(q, k, v, g, S0)
    o2, S2 = linear_forward(q[:, :, 3:], k[:, :, 3:], v[:, :, 3:], g[:, :, 3:])
    np.testing.assert_array_equal(o[:, :, 3:], o2)
    np.testing.assert_array_equal(S, S2)


def test_shared_heads_read_their_own_group():
    q, k, v, g, S0 = _draw(np.random.default_rng(3), H=6, Hqk=2)
    o, _ = linear_forward(q, k, v, g, S0)
    for h in range(6):
        one, _ = linear_forward(q[:, h // 3:h // 3 + 1], k[:, h // 3:h // 3 + 1], v[:, h:h + 1],
                                g[:, h:h + 1], S0[:, h:h + 1])
        np.testing.assert_array_equal(o[:, h:h + 1], one)


@pytest.mark.parametrize("groups", [1, 3])
def test_backward_is_the_difference_quotient(groups):
    rng = np.random.default_rng(4)
    q, k, v, g, S0 = _draw(rng, H=2 * groups, L=5)
    dO, dS = rng.standard_normal(v.shape), rng.standard_normal(S0.shape)
    x = [q, k, v, g, S0]

    def loss():
        o, S = linear_forward(*x)
        return (o * dO).sum() + (S * dS).sum()

    for a, d in zip(x, linear_backward(q, k, v, g, S0, dO, dS)):
        num = np.zeros_like(a)
        for i in np.ndindex(a.shape):
            keep, h = a[i], 1e-5
            a[i] = keep + h
            up = loss()
            a[i] = keep - h
            num[i] = (up - loss()) / (2 * h)
            a[i] = keep
        np.testing.assert_allclose(d, num, rtol=1e-7, atol=1e-8)


def test_rotation_by_hand():
    x = np.arange(1.0, 9.0).reshape(1, 1, 1, 8)
    quarter = np.full((1, 1, 2), np.pi / 2)
    np.testing.assert_allclose(rotate(x, quarter)[0, 0, 0], [-3, -4, 1, 2, 5, 6, 7, 8], atol=1e-12)
    np.testing.assert_allclose(rotate(x, quarter, interleaved=True)[0, 0, 0],
                               [-2, 1, -4, 3, 5, 6, 7, 8], atol=1e-12)
    np.testing.assert_allclose(rotate(rotate(x, quarter), quarter, inverse=True), x, atol=1e-12)


def test_angles_by_axis():
    pos = np.array([[[3, 4]], [[50, 60]]])  # two axes, one row of two tokens
    a = rotation_angles(pos, [1.0, 0.5, 0.25], [1, 2])
    np.testing.assert_allclose(a, [[[3, 25, 12.5], [4, 30, 15]]])


def test_product_of_rotated_rows_depends_on_the_distance():
    rng = np.random.default_rng(5)
    q, k = rng.standard_normal((2, 1, 1, 1, 8))
    f = [1.0, 0.3, 0.1, 0.01]
    at = lambda x, p: norm_rope(x, None, rotation_angles([[p]], f))  # noqa: E731
    np.testing.assert_allclose((at(q, 9) * at(k, 4)).sum(), (at(q, 105) * at(k, 100)).sum(),
                               rtol=1e-12)


def test_norm_has_unit_mean_square():
    x = np.random.default_rng(6).standard_normal((1, 2, 3, 64)) * 7
    y = norm_rope(x, None, rotation_angles(np.arange(3)[None], np.ones(8)), eps=0.0)
    np.testing.assert_allclose((y * y).mean(-1), 1.0, rtol=1e-12)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("norm", [False, True])
def test_norm_rope_backward_is_the_difference_quotient(norm, interleaved):
    rng = np.random.default_rng(7)
    x, w = rng.standard_normal((1, 2, 3, 8)), rng.standard_normal(8)
    a = rotation_angles(rng.integers(0, 50, (2, 1, 3)), [1.0, 0.3, 0.1], [1, 2])
    dy = rng.standard_normal(x.shape)
    got = norm_rope_backward(x, w, a, dy, 1e-3, norm, interleaved)
    for t, d in zip((x, w), got):
        num = np.zeros_like(t)
        for i in np.ndindex(t.shape):
            keep, h = t[i], 1e-5
            t[i] = keep + h
            up = (norm_rope(x, w, a, 1e-3, norm, interleaved) * dy).sum()
            t[i] = keep - h
            num[i] = (up - (norm_rope(x, w, a, 1e-3, norm, interleaved) * dy).sum()) / (2 * h)
            t[i] = keep
        np.testing.assert_allclose(d, num, rtol=1e-7, atol=1e-8)
