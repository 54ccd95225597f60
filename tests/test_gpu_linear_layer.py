"""The operators as a layer runs them: norm and rotation of a fused
projection's q and k, the gated linear recurrence over a prompt, its gradients
back to the projection, and single tokens from the prompt's state."""

import numpy as np
import pytest
import torch

from deltanet_delta_rule_chunk_amd import binding as N
from oracle import (linear_backward, linear_forward, norm_rope,
                    norm_rope_backward, rotation_angles)
from parity import to64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _layer(seed, B, Hqk, grp, L, d, dt):
    rng = np.random.default_rng(seed)
    t = torch.bfloat16 if dt == "bf16" else torch.float32
    H = Hqk * grp
    proj = torch.from_numpy(rng.standard_normal((B, L, 2 * Hqk + H, d))).to(t).to(DEV)
    w = torch.from_numpy(d ** -0.5 * (1 + 0.2 * rng.standard_normal(d))).float().to(DEV)
    g = torch.nn.functional.logsigmoid(torch.from_numpy(rng.standard_normal((B, H, L)) + 3)).float().to(DEV)
    pos = torch.arange(L, device=DEV, dtype=torch.int32).expand(B, L).contiguous() + 1000
    inv = torch.from_numpy(10000.0 ** (-np.arange(d // 2) / (d // 2))).float().to(DEV)
    dO = torch.from_numpy(rng.standard_normal((B, H, L, d))).to(t).to(DEV)
    return proj, w, g, pos, inv, dO


@pytest.mark.parametrize("dt,B,Hqk,grp,L,d", [("f32", 2, 2, 2, 200, 64), ("bf16", 1, 2, 1, 330, 128)])
def test_training_step(gpu_lib, dt, B, Hqk, grp, L, d):
    proj, w, g, pos, inv, dO = _layer(1, B, Hqk, grp, L, d, dt)
    leaves = [proj.requires_grad_(), w.requires_grad_(), g.requires_grad_()]
    part = lambda a, b: proj[:, :, a:b].transpose(1, 2)  # noqa: E731
    q, k = N.rotary_qk(part(0, Hqk), part(Hqk, 2 * Hqk), pos, inv, k_weight=w)
    v = part(2 * Hqk, 2 * Hqk + Hqk * grp).contiguous()
    o, _ = N.linear_rule(q, k, v, g)
    dproj, dw, dg = torch.autograd.grad(o, leaves, dO)

    p, a = to64(proj), rotation_angles(to64(pos), to64(inv))
    cut = lambda x, y: p[:, :, x:y].transpose(0, 2, 1, 3)  # noqa: E731
    q64, k64 = norm_rope(cut(0, Hqk), None, a), norm_rope(cut(Hqk, 2 * Hqk), to64(w), a)
    v64 = cut(2 * Hqk, p.shape[2])
    o64, _ = linear_forward(q64, k64, v64, to64(g))
    dq, dk, dv, dg64, _ = linear_backward(q64, k64, v64, to64(g), None, to64(dO))
    dqr, _ = norm_rope_backward(cut(0, Hqk), None, a, dq)
    dkr, dw64 = norm_rope_backward(cut(Hqk, 2 * Hqk), to64(w), a, dk)
    dp64 = np.concatenate([dqr, dkr, dv], 1).transpose(0, 2, 1, 3)
    # Norms of differences.  bf16: q_hat, k_hat, then their gradients and the
    # result are rounded, 2^-8 each at most and in the mean a fraction of it:
    # five roundings.  fp32: sums of L + 512 terms.
    tol = 5 * 2.0 ** -8 if dt == "bf16" else (L + 512) * 2.0 ** -24
    for got, want in ((o, o64), (dproj, dp64), (dw, dw64), (dg, dg64)):
        assert np.linalg.norm(to64(got) - want) <= tol * np.linalg.norm(want)


def test_prompt_then_single_tokens(gpu_lib):
    B, Hqk, grp, L, d, P = 2, 2, 2, 90, 64, 83
    proj, w, g, pos, inv, _ = _layer(2, B, Hqk, grp, L, d, "f32")
    H = Hqk * grp

    def rows(a, b):
        x = proj[:, a:b]
        q, k = N.qk_norm_rope(x[:, :, :Hqk].transpose(1, 2), x[:, :, Hqk:2 * Hqk].transpose(1, 2),
                              pos[:, a:b].contiguous(), inv, k_weight=w)
        return q, k, x[:, :, 2 * Hqk:].transpose(1, 2).contiguous(), g[:, :, a:b].contiguous()

    whole, S_whole = N.linear_chunk_fwd(*rows(0, L))
    o, S = N.linear_chunk_fwd(*rows(0, P))
    outs = [o]
    for t in range(P, L):
        one = [x[:, :, 0] for x in rows(t, t + 1)]
        outs.append(N.linear_decode_step(*one, S)[:, :, None])
    got = torch.cat(outs, 2)
    scale = float(whole.abs().max())
    assert float((got - whole).abs().max()) <= (L + 512) * 2.0 ** -24 * 8 * scale
    assert float((S - S_whole).abs().max()) <= (L + 512) * 2.0 ** -24 * 8 * float(S_whole.abs().max())
    q, k, v, gg = (to64(x) for x in rows(0, L))
    want, S64 = linear_forward(q, k, v, gg)
    assert np.linalg.norm(to64(got) - want) <= (L + 512) * 2.0 ** -24 * np.linalg.norm(want)
    assert got.shape == (B, H, L, d)
