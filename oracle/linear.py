"""Plain fp64 gated linear recurrence: forward, decode step and backward.

Per (b, h) and token t, in order: ``S = e^{g_t} S + k_t^T v_t``, ``o_t = q_t S``.
State head h reads q and k of head ``h // (H / H_qk)``.
"""

from __future__ import annotations

import numpy as np


def _heads(x, H):
    return np.repeat(x, H // x.shape[1], axis=1)


def _decay(g):
    with np.errstate(invalid="ignore"):
        return np.exp(np.asarray(g, dtype=np.float64))


def linear_decode_step(q, k, v, g, S):
    """One token: q, k ``[B,H_qk,d_k]``, v ``[B,H,d_v]``, g ``[B,H]`` or None,
    S ``[B,H,d_k,d_v]``; returns (o, new S)."""
    H = v.shape[1]
    q, k = _heads(q, H), _heads(k, H)
    a = 1.0 if g is None else _decay(g)[..., None, None]
    S = a * S + k[..., :, None] * v[..., None, :]
    return np.einsum("bhk,bhkv->bhv", q, S), S


def linear_forward(q, k, v, g=None, S0=None):
    """The recurrence over L tokens; returns (o, S_final)."""
    B, H, L, dv = v.shape
    S = np.zeros((B, H, q.shape[-1], dv)) if S0 is None else np.array(S0, dtype=np.float64)
    o = np.zeros((B, H, L, dv))
    for t in range(L):
        o[:, :, t], S = linear_decode_step(q[:, :, t], k[:, :, t], v[:, :, t],
                                           None if g is None else g[:, :, t], S)
    return o, S


def linear_backward(q, k, v, g, S0, dO, dS_final=None):
    """Gradients (dq, dk, dv, dg, dS0) by the token loop backwards over kept
    states; dg is None without g."""
    B, H, L, dv_ = v.shape
    H_qk, dk_ = q.shape[1], q.shape[-1]
    qe, ke = _heads(q, H), _heads(k, H)
    S = np.zeros((B, H, dk_, dv_)) if S0 is None else np.array(S0, dtype=np.float64)
    states = [S]
    for t in range(L):
        _, S = linear_decode_step(q[:, :, t], k[:, :, t], v[:, :, t],
                                  None if g is None else g[:, :, t], S)
        states.append(S)
    G = np.zeros_like(S) if dS_final is None else np.array(dS_final, dtype=np.float64)
    dq, dk, dv = np.zeros_like(qe), np.zeros_like(ke), np.zeros((B, H, L, dv_))
    dg = None if g is None else np.zeros((B, H, L))
    for t in range(L - 1, -1, -1):
        G = G + qe[:, :, t, :, None] * dO[:, :, t, None, :]
        dq[:, :, t] = np.einsum("bhkv,bhv->bhk", states[t + 1], dO[:, :, t])
        dk[:, :, t] = np.einsum("bhkv,bhv->bhk", G, v[:, :, t])
        dv[:, :, t] = np.einsum("bhkv,bhk->bhv", G, ke[:, :, t])
        if g is not None:
            a = _decay(g[:, :, t])
            dg[:, :, t] = a * np.einsum("bhkv,bhkv->bh", states[t], G)
            G = a[..., None, None] * G
    share = lambda x: x.reshape(B, H_qk, H // H_qk, L, dk_).sum(2)  # noqa: E731
    return share(dq), share(dk), dv, dg, G
