"""Plain fp64 per-head RMS norm and rotation by position, and its gradient."""

from __future__ import annotations

import numpy as np


def rotation_angles(positions, inv_freq, sections=None):
    """``[B, L, pairs]`` angles: positions ``[axes, B, L]`` (or ``[B, L]``)."""
    p = np.asarray(positions, dtype=np.float64)
    p = p[None] if p.ndim == 2 else p
    sections = [len(inv_freq)] if sections is None else sections
    axis = np.repeat(np.arange(len(sections)), sections)
    return np.moveaxis(p[axis], 0, -1) * np.asarray(inv_freq, dtype=np.float64)


def rotate(x, angles, interleaved=False, inverse=False):
    """x ``[B, H, L, d]``; pair j of its first ``2 * pairs`` elements turned by
    ``angles[..., j]``, one 2 x 2 matrix per pair."""
    n = angles.shape[-1]
    y = np.array(x, dtype=np.float64)
    c, s = np.cos(angles)[:, None], np.sin(angles)[:, None] * (-1 if inverse else 1)
    for j in range(n):
        ia, ib = (2 * j, 2 * j + 1) if interleaved else (j, j + n)
        a, b = x[..., ia], x[..., ib]
        y[..., ia] = a * c[..., j] - b * s[..., j]
        y[..., ib] = a * s[..., j] + b * c[..., j]
    return y


def norm_rope(x, weight, angles, eps=1e-6, norm=True, interleaved=False):
    """``rotate(x / sqrt(mean(x^2) + eps) * weight)`` (no division without norm)."""
    x = np.asarray(x, dtype=np.float64)
    n = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps) if norm else x
    n = n if weight is None else n * weight
    return rotate(n, angles, interleaved)


def norm_rope_backward(x, weight, angles, dy, eps=1e-6, norm=True, interleaved=False):
    """(dx, dweight) by the chain rule: with s = mean(x^2) + eps, n_i = x_i s^{-1/2},
    d n_i / d x_j = delta_ij s^{-1/2} - x_i x_j s^{-3/2} / d."""
    x = np.asarray(x, dtype=np.float64)
    d = x.shape[-1]
    dn = rotate(dy, angles, interleaved, inverse=True)
    w = np.ones(d) if weight is None else np.asarray(weight, dtype=np.float64)
    if not norm:
        return dn * w, (dn * x).sum((0, 1, 2))
    s = np.mean(x * x, -1, keepdims=True) + eps
    u = dn * w
    dx = u * s ** -0.5 - x * (x * u).sum(-1, keepdims=True) * s ** -1.5 / d
    return dx, (dn * x * s ** -0.5).sum((0, 1, 2))
