"""The plain state space layer's operators against other forms of their formulas,
and their gradients against differences."""

import numpy as np
import pytest

from oracle import (add_norm, add_norm_backward, conv_backward, conv_forward, scan_backward, scan_forward,
                    spans_of)

STEP = 1e-6


def _differences(f, x, pick, rng):
    """(place, derivative of f by central differences) at some places of x."""
    for _ in range(pick):
        at = tuple(rng.integers(0, n) for n in x.shape)
        old = x[at]
        x[at] = old + STEP
        hi = f()
        x[at] = old - STEP
        lo = f()
        x[at] = old
        yield at, (hi - lo) / (2 * STEP)


def _near(got, want, magnitude=0.0):
    """A difference of two sums of terms that add up to `magnitude` is itself off by a few
    roundings (2^-53) of that, divided by the step."""
    quotient = 4 * 2.0 ** -53 * magnitude / STEP
    assert abs(got - want) <= 2e-7 * (1 + abs(want)) + quotient, (got, want)


SPANS = {"batch": (2, 9, None), "packed": (1, 14, [2, 7, 7, 8, 12]), "short": (1, 4, [0, 1, 3, 4])}


@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("where", SPANS)
@pytest.mark.parametrize("silu", [True, False])
def test_conv_gradients(K, where, silu):
    B, L, cu = SPANS[where]
    spans = spans_of(B, L, cu)
    rng = np.random.default_rng(K)
    x, w, b = rng.normal(size=(B, L, 5)), rng.normal(size=(5, K)), rng.normal(size=5)
    s0 = rng.normal(size=(len(spans), K - 1, 5))
    dy, dstate = rng.normal(size=x.shape), rng.normal(size=s0.shape)

    def loss():
        y, s = conv_forward(x, w, b, s0, spans, silu)
        return (y * dy).sum() + (s * dstate).sum()

    grads = conv_backward(x, w, b, s0, dy, dstate, spans, silu)
    for v, g in zip((x, w, b, s0), grads):
        for at, d in _differences(loss, v, 12, rng):
            _near(g[at], d)


@pytest.mark.parametrize("where", SPANS)
@pytest.mark.parametrize("gate,softplus", [(True, True), (False, False)])
def test_scan_gradients(where, gate, softplus):
    B, L, cu = SPANS[where]
    spans = spans_of(B, L, cu)
    rng = np.random.default_rng(7)
    D, N = 3, 4
    u, dt, z = (rng.normal(size=(B, L, D)) for _ in range(3))
    if not softplus:
        dt = np.abs(dt)
    A, Bm, Cm = -np.exp(rng.normal(size=(D, N))), rng.normal(size=(B, L, N)), rng.normal(size=(B, L, N))
    skip, bias = rng.normal(size=D), rng.normal(size=D)
    h0 = rng.normal(size=(len(spans), D, N))
    dy, dh = rng.normal(size=u.shape), rng.normal(size=h0.shape)
    how = dict(D=skip, z=z if gate else None, dt_bias=bias, h0=h0, softplus=softplus)

    def loss():
        y, h = scan_forward(u, dt, A, Bm, Cm, spans, **how)
        return (y * dy).sum() + (h * dh).sum()

    ym, hm = scan_forward(u, dt, A, Bm, Cm, spans, **how, size=True)
    magnitude = (ym * np.abs(dy)).sum() + (hm * np.abs(dh)).sum()
    grads = scan_backward(u, dt, A, Bm, Cm, dy, dh, spans, **how)
    for v, g in zip((u, dt, A, Bm, Cm, skip, z, bias, h0), grads):
        if v is z and not gate:
            continue
        for at, d in _differences(loss, v, 10, rng):
            _near(g[at], d, magnitude)


def test_scan_in_closed_form():
    """One state of one channel at a constant step: a geometric sum."""
    L, step, a = 20, 0.3, -0.7
    one = np.ones((1, L, 1))
    y, h = scan_forward(one, one * step, np.array([[a]]), one, one, spans_of(1, L), softplus=False)
    q = np.exp(a * step)
    want = step * (1 - q ** np.arange(1, L + 1)) / (1 - q)
    assert np.allclose(y[0, :, 0], want, rtol=1e-13) and np.isclose(h[0, 0, 0], want[-1], rtol=1e-13)


def test_pieces_of_a_sequence_make_the_whole():
    rng = np.random.default_rng(3)
    x, w = rng.normal(size=(1, 11, 4)), rng.normal(size=(4, 4))
    whole, kept = conv_forward(x, w, None, None, spans_of(1, 11))
    s, parts = None, []
    for lo, hi in ((0, 1), (1, 2), (2, 9), (9, 11)):
        y, s = conv_forward(x[:, lo:hi], w, None, s, spans_of(1, hi - lo))
        parts.append(y)
    assert np.allclose(np.concatenate(parts, 1), whole, atol=1e-15) and np.array_equal(s, kept)


def test_norm_gradient():
    rng = np.random.default_rng(5)
    total, w = rng.normal(size=(3, 6)), rng.normal(size=6)
    dy, dt = rng.normal(size=total.shape), rng.normal(size=total.shape)
    loss = lambda: (add_norm(total, w, 1e-3) * dy).sum() + (total * dt).sum()  # noqa: E731
    d, dw = add_norm_backward(total, w, dy, dt, 1e-3)
    for v, g in ((total, d), (w, dw)):
        for at, num in _differences(loss, v, 12, rng):
            _near(g[at], num)
