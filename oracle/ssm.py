"""Plain fp64 operators of a state space layer: the short causal convolution, the
selective scan, the norm with the residual's addition, and their gradients.

Sequences are given as ``spans``, (batch row, first token, one behind the last)
of each; the states' leading index counts them.  Rows that no span holds are zeros.

``size=True`` evaluates the same sums with every term's magnitude, for bounds on
rounding errors.
"""

from __future__ import annotations

import numpy as np


def spans_of(B, L, cu=None):
    if cu is None:
        return [(b, 0, L) for b in range(B)]
    return [(0, int(lo), int(hi)) for lo, hi in zip(cu[:-1], cu[1:])]


def _sigmoid(x):
    with np.errstate(over="ignore"):
        return 1.0 / (1.0 + np.exp(-x))


def _silu(x):
    return x * _sigmoid(x)


def _dsilu(x):
    s = _sigmoid(x)
    return s * (1.0 + x * (1.0 - s))


# ---- short convolution ---------------------------------------------------------------


def _extended(x, state0, K, i, span):
    row, lo, hi = span
    front = np.zeros((K - 1, x.shape[2])) if state0 is None else state0[i]
    return np.concatenate([front, x[row, lo:hi]])


def _tap_sums(e, w, b, n):
    K = w.shape[1]
    p = sum(w[:, j] * e[j:j + n] for j in range(K))
    return p if b is None else p + b


def conv_forward(x, weight, bias, state0, spans, silu=True):
    """(y, kept rows)."""
    K = weight.shape[1]
    y, state = np.zeros(x.shape), np.zeros((len(spans), K - 1, x.shape[2]))
    for i, (row, lo, hi) in enumerate(spans):
        e = _extended(x, state0, K, i, (row, lo, hi))
        p = _tap_sums(e, weight, bias, hi - lo)
        y[row, lo:hi] = _silu(p) if silu else p
        state[i] = e[hi - lo:]
    return y, state


def conv_backward(x, weight, bias, state0, dy, dstate, spans, silu=True, size=False):
    """(dx, dweight, dbias, dstate0)."""
    K = weight.shape[1]
    D = x.shape[2]
    m = np.abs if size else (lambda v: v)
    dx, dw, db = np.zeros(x.shape), np.zeros(weight.shape), np.zeros(D)
    ds = np.zeros((len(spans), K - 1, D))
    for i, (row, lo, hi) in enumerate(spans):
        n = hi - lo
        e = _extended(x, state0, K, i, (row, lo, hi))
        q = dy[row, lo:hi]
        if silu:
            p = _tap_sums(e, weight, bias, n)
            if size:  # silu' and what the tap sums' rounding does to it (|silu''| <= 1/2)
                pm = _tap_sums(np.abs(e), np.abs(weight), None if bias is None else np.abs(bias), n)
                q = np.abs(q) * (1.1 + 0.5 * pm)
            else:
                q = q * _dsilu(p)
        q = m(q)
        de = np.zeros(e.shape)
        if dstate is not None:
            de[n:] += m(dstate[i])
        for j in range(K):
            de[j:j + n] += m(weight[:, j]) * q
            dw[:, j] += (q * m(e[j:j + n])).sum(0)
        db += q.sum(0)
        ds[i], dx[row, lo:hi] = de[:K - 1], de[K - 1:]
    return dx, dw, db, ds


# ---- selective scan --------------------------------------------------------------------


def _steps(dt, dt_bias, softplus):
    raw = dt if dt_bias is None else dt + dt_bias
    return (np.logaddexp(raw, 0.0) if softplus else raw), raw


def scan_forward(u, dt, A, B, C, spans, D=None, z=None, dt_bias=None, h0=None, softplus=True,
                 size=False):
    """(y, last states)."""
    m = np.abs if size else (lambda v: v)
    s, _ = _steps(dt, dt_bias, softplus)
    width, N = A.shape
    y = np.zeros(u.shape)
    hT = np.zeros((len(spans), width, N))
    for i, (row, lo, hi) in enumerate(spans):
        h = np.zeros((width, N)) if h0 is None else m(h0[i])
        for t in range(lo, hi):
            h = np.exp(s[row, t, :, None] * A) * h + m(s[row, t] * u[row, t])[:, None] * m(B[row, t])
            y[row, t] = (h * m(C[row, t])).sum(-1)
            if D is not None:
                y[row, t] += m(D * u[row, t])
            if z is not None:
                y[row, t] *= m(_silu(z[row, t]))
        hT[i] = h
    return y, hT


def scan_backward(u, dt, A, B, C, dy, dhT, spans, D=None, z=None, dt_bias=None, h0=None,
                  softplus=True, size=False):
    """(du, ddt, dA, dB, dC, dD, dz, ddt_bias, dh0)."""
    m = np.abs if size else (lambda v: v)
    s, raw = _steps(dt, dt_bias, softplus)
    slope = _sigmoid(raw) if softplus else np.ones(raw.shape)
    width, N = A.shape
    du, ddt, dz = np.zeros(u.shape), np.zeros(u.shape), np.zeros(u.shape)
    dB, dC, dA = np.zeros(B.shape), np.zeros(C.shape), np.zeros(A.shape)
    dD, db = np.zeros(width), np.zeros(width)
    dh0 = np.zeros((len(spans), width, N))
    skip = np.zeros(width) if D is None else D
    for i, (row, lo, hi) in enumerate(spans):
        h = np.zeros((width, N)) if h0 is None else m(h0[i])
        before = []
        for t in range(lo, hi):
            before.append(h)
            h = np.exp(s[row, t, :, None] * A) * h + m(s[row, t] * u[row, t])[:, None] * m(B[row, t])
        G = np.zeros((width, N)) if dhT is None else m(dhT[i])
        for t in range(hi - 1, lo - 1, -1):
            a = np.exp(s[row, t, :, None] * A)
            x = m(s[row, t] * u[row, t])
            ht = a * before[t - lo] + x[:, None] * m(B[row, t])
            g = m(dy[row, t])
            if z is not None:
                plain = (ht * m(C[row, t])).sum(-1) + m(skip * u[row, t])
                dz[row, t] = g * plain * (1.1 if size else _dsilu(z[row, t]))
                g = g * m(_silu(z[row, t]))
            G = G + m(C[row, t]) * g[:, None]
            dC[row, t] = (ht * g[:, None]).sum(0)
            dB[row, t] = (G * x[:, None]).sum(0)
            dx = (G * m(B[row, t])).sum(-1)
            through = G * a * before[t - lo]
            ds = (through * m(A)).sum(-1) + dx * m(u[row, t])
            dA += through * m(s[row, t])[:, None]
            du[row, t] = dx * m(s[row, t]) + m(skip) * g
            ddt[row, t] = ds * slope[row, t]
            dD += g * m(u[row, t])
            db += ddt[row, t]
            G = G * a
        dh0[i] = G
    return du, ddt, dA, dB, dC, dD, dz, db, dh0


# ---- norm with addition -----------------------------------------------------------------


def add_norm(total, weight, eps):
    """y of the rows that x + residual rounds to."""
    return total / np.sqrt((total ** 2).mean(-1, keepdims=True) + eps) * weight


def add_norm_backward(total, weight, dy, dtotal, eps):
    """(gradient of x and of the residual, dweight)."""
    r = 1.0 / np.sqrt((total ** 2).mean(-1, keepdims=True) + eps)
    n, v = total * r, dy * weight
    d = r * (v - n * (n * v).mean(-1, keepdims=True))
    return (d if dtotal is None else d + dtotal), (dy * n).reshape(-1, total.shape[-1]).sum(0)
