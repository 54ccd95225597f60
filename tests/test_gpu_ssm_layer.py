"""The operators as a state space layer runs them: norm with the residual's addition,
in-projection, convolution, the projections of the steps, B and C, the scan with its
gate, out-projection; a training step, packed documents, a prompt and its next tokens,
and a decode step in a graph.

Bounds on norms of differences: fp32 (L + 1024) roundings of 2^-24 (the longest sums are
over L tokens, and 128 channels a few times); bf16: 7 tensors between the operators are
rounded on the way there and 7 on the way back, 2^-8 each at most.
"""

import numpy as np
import pytest
import torch
import torch.nn.functional as F

from deltanet_delta_rule_chunk_amd import binding as N
from oracle import spans_of

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
D, E, R, S, K = 64, 128, 8, 16, 4
EPS = 1e-5


def _params(seed, t):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, std=1.0: torch.randn(s, generator=g) * std  # noqa: E731
    start = torch.exp(torch.rand((E,), generator=g) * 4.6 - 6.9)
    p = dict(norm=1 + r(D, std=0.2), W_in=r(2 * E, D, std=D ** -0.5).to(t), conv=r(E, K, std=0.5), conv_b=r(E, std=0.1),
             W_x=r(R + 2 * S, E, std=E ** -0.5).to(t), W_dt=r(E, R, std=R ** -0.5).to(t),
             dt_b=start + torch.log(-torch.expm1(-start)), A=-torch.arange(1, S + 1) * torch.exp(r(E, S, std=0.1)),
             skip=1 + r(E, std=0.1), W_out=r(D, E, std=E ** -0.5).to(t))
    return p


def _layer(p, x, res, kept=None, h0=None, cu=None):
    """As a user's program writes it; differentiable."""
    y, total = N.residual_norm(x, res, p["norm"], eps=EPS)
    rows = y @ p["W_in"].t()
    c, kept = N.short_conv(rows[..., :E], p["conv"], p["conv_b"], kept, cu_seqlens=cu)
    few = c @ p["W_x"].t()
    s, h = N.selective_scan(c, few[..., :R] @ p["W_dt"].t(), p["A"], few[..., R:R + S], few[..., R + S:], D=p["skip"],
                            z=rows[..., E:], dt_bias=p["dt_b"], h0=h0, cu_seqlens=cu)
    return s @ p["W_out"].t(), total, kept, h


def _token(p, x, res, kept, h):
    """One token of every sequence; kept and h are updated."""
    y, total = N.add_rms_norm(x, res, p["norm"], eps=EPS)
    rows = y @ p["W_in"].t()
    c = N.short_conv_step(rows[..., :E], p["conv"], p["conv_b"], kept)
    few = c @ p["W_x"].t()
    s = N.selective_scan_step(c, few[..., :R] @ p["W_dt"].t(), p["A"], few[..., R:R + S], few[..., R + S:], h, D=p["skip"],
                              z=rows[..., E:], dt_bias=p["dt_b"])
    return s @ p["W_out"].t(), total


def _plain(p, x, res, kept, h0, spans):
    """The same in fp64 on the CPU, with torch's gradients."""
    total = x + res
    y = total / torch.sqrt((total ** 2).mean(-1, keepdim=True) + EPS) * p["norm"]
    rows = y @ p["W_in"].t()
    xin, z = rows[..., :E], rows[..., E:]
    out, ends, states = torch.zeros(*x.shape[:2], E, dtype=torch.float64), [], []
    parts = {}
    for i, (b, lo, hi) in enumerate(spans):
        e = torch.cat([kept[i], xin[b, lo:hi]])
        ends.append(e[hi - lo:])
        c = F.silu(sum(p["conv"][:, j] * e[j:j + hi - lo] for j in range(K)) + p["conv_b"])
        few = c @ p["W_x"].t()
        dt = F.softplus(few[:, :R] @ p["W_dt"].t() + p["dt_b"])
        h, ys = h0[i], []
        for t in range(hi - lo):
            h = torch.exp(dt[t, :, None] * p["A"]) * h + (dt[t] * c[t])[:, None] * few[t, R:R + S]
            ys.append((h * few[t, R + S:]).sum(-1) + p["skip"] * c[t])
        states.append(h)
        if ys:
            parts[i] = torch.stack(ys) * F.silu(z[b, lo:hi])
    for i, (b, lo, hi) in enumerate(spans):
        if i in parts:
            out[b, lo:hi] = parts[i]
    return out @ p["W_out"].t(), total, torch.stack(ends), torch.stack(states)


def _near(got, want, tol, what):
    d, n = float((got.detach().double().cpu() - want.detach()).norm()), float(want.detach().norm())
    assert d <= tol * n, (what, d / n, tol)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("B,L,cu", [(2, 70, None), (1, 150, [0, 40, 40, 41, 144])])
def test_training_step(gpu_lib, dtype, B, L, cu):
    p = _params(1, dtype)
    g = torch.Generator().manual_seed(2)
    n = B if cu is None else len(cu) - 1
    r = lambda *s, t=dtype: torch.randn(s, generator=g).to(t)  # noqa: E731
    x, res, dout, dtotal = r(B, L, D), r(B, L, D, t=torch.float32), r(B, L, D), r(B, L, D, t=torch.float32)
    kept, h0 = r(n, K - 1, E), r(n, E, S, t=torch.float32)
    gp = {k: v.to(DEV).requires_grad_() for k, v in p.items()}
    leaves = [t.to(DEV).requires_grad_() for t in (x, res, kept, h0)]
    cut = None if cu is None else torch.tensor(cu, dtype=torch.int32, device=DEV)
    got = _layer(gp, *leaves, cut)
    dgot = torch.autograd.grad([got[0], got[1]], [*gp.values(), *leaves], [dout.to(DEV), dtotal.to(DEV)])
    wp = {k: v.double().requires_grad_() for k, v in p.items()}
    wl = [t.double().requires_grad_() for t in (x, res, kept, h0)]
    want = _plain(wp, *wl, spans_of(B, L, cu))
    dwant = torch.autograd.grad([want[0], want[1]], [*wp.values(), *wl], [dout.double(), dtotal.double()])
    tol = 14 * 2.0 ** -8 if dtype == torch.bfloat16 else (L + 1024) * 2.0 ** -24
    for a, b, what in zip(got, want, ("out", "total", "kept", "h")):
        _near(a, b, tol, what)
    for a, b, what in zip(dgot, dwant, (*p, "x", "residual", "kept", "h0")):
        _near(a, b, tol, "d " + what)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_prompts_then_single_tokens(gpu_lib, dtype):
    """Packed prompts of different lengths, then tokens of all of them at once, against the
    whole sequences in one call each."""
    p = {k: v.to(DEV) for k, v in _params(3, dtype).items()}
    g = torch.Generator().manual_seed(4)
    lengths, more = [37, 1, 64, 90], 6
    xs = [torch.randn((n + more, D), generator=g).to(dtype).to(DEV) for n in lengths]
    rs = [torch.randn((n + more, D), generator=g).to(DEV) for n in lengths]
    cut = torch.tensor(np.cumsum([0, *lengths]), dtype=torch.int32, device=DEV)
    first = lambda v: torch.cat([a[:n] for a, n in zip(v, lengths)])[None]  # noqa: E731
    out, _, kept, h = _layer(p, first(xs), first(rs), cu=cut)
    outs = [[out[0, cut[i]:cut[i + 1]]] for i in range(len(lengths))]
    for t in range(more):
        at = lambda v: torch.stack([a[n + t] for a, n in zip(v, lengths)])  # noqa: E731
        o, _ = _token(p, at(xs), at(rs), kept, h)
        for i in range(len(lengths)):
            outs[i].append(o[i:i + 1])
    tol = 7 * 2.0 ** -8 if dtype == torch.bfloat16 else (96 + 1024) * 2.0 ** -24
    for i, (x, r) in enumerate(zip(xs, rs)):
        want, _, k1, h1 = _layer(p, x[None], r[None])
        _near(torch.cat(outs[i]), want[0].double().cpu(), tol, "out")
        _near(h[i], h1[0].double().cpu(), tol, "h")
        _near(kept[i], k1[0].double().cpu(), tol, "kept")


def test_decode_in_a_graph(gpu_lib):
    """A token of a layer captured once and replayed on new inputs, with eager work between."""
    p = {k: v.to(DEV) for k, v in _params(5, torch.bfloat16).items()}
    B = 3
    x, res = torch.zeros((B, D), device=DEV, dtype=torch.bfloat16), torch.zeros((B, D), device=DEV)
    kept, h = torch.zeros((B, K - 1, E), device=DEV, dtype=torch.bfloat16), torch.zeros((B, E, S), device=DEV)
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        for _ in range(3):
            _token(p, x, res, kept, h)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, total = _token(p, x, res, kept, h)
    kept.zero_(), h.zero_()
    k2, h2 = kept.clone(), h.clone()
    for i in range(5):
        x.copy_(torch.randn((B, D), device=DEV))
        res.copy_(torch.randn((B, D), device=DEV))
        graph.replay()
        want, t2 = _token(p, x, res, k2, h2)
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(total, t2) and torch.equal(kept, k2) and torch.equal(h, h2), i


def test_sequences_in_a_graph(gpu_lib):
    """Forward and backward calls of packed sequences captured once; other inputs and other
    cuts between the replays."""
    p = {k: v.to(DEV) for k, v in _params(6, torch.float32).items()}
    L, n = 200, 4
    cu = torch.tensor([0, 50, 60, 130, 190], dtype=torch.int32, device=DEV)
    u, dt, z, dy = (torch.randn((1, L, E), device=DEV) for _ in range(4))
    Bm, Cm = torch.randn((1, L, S), device=DEV), torch.randn((1, L, S), device=DEV)
    h0, kept = torch.randn((n, E, S), device=DEV), torch.randn((n, K - 1, E), device=DEV)
    how = dict(D=p["skip"], z=z, dt_bias=p["dt_b"], h0=h0, cu_seqlens=cu)

    def calls():
        return [t for t in (*N.short_conv_fwd(u, p["conv"], p["conv_b"], kept, cu_seqlens=cu),
                            *N.short_conv_bwd(u, p["conv"], p["conv_b"], kept, dy, kept, cu_seqlens=cu),
                            *N.selective_scan_fwd(u, dt, p["A"], Bm, Cm, **how),
                            *N.selective_scan_bwd(u, dt, p["A"], Bm, Cm, dy, h0, **how),
                            *N.add_rms_norm(u, z, p["skip"]), *N.add_rms_norm_fp8(u, z, p["skip"])[:2],
                            *N.add_rms_norm_bwd(u, p["skip"], dy, z)) if t is not None]

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        calls()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = calls()
    for cuts in ([0, 50, 60, 130, 190], [0, 0, 0, 200, 200], [3, 4, 100, 101, 102], [0, 50, 60, 130, 190]):
        for t in (u, dt, z, dy, Bm, Cm):
            t.normal_()
        cu.copy_(torch.tensor(cuts, dtype=torch.int32))
        graph.replay()
        want = calls()
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            a, b = (t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for t in (a, b))
            assert torch.equal(a, b), (cuts, i)
