"""The gated linear recurrence and the q / k norm with rotation at the ends of
what their documentation allows: tensors past 2^31 elements, the most heads,
calls under way at once, a gradient of a gradient.  Bounds: those of
test_gpu_linear and test_gpu_qk_norm_rope."""

import threading

import numpy as np
import pytest
import torch

from deltanet_delta_rule_chunk_amd import binding as N
from oracle import linear_backward, linear_forward, norm_rope, norm_rope_backward, rotation_angles
from parity import to64
from test_gpu_linear import _close, _gpu, _inputs, _np
from test_gpu_qk_norm_rope import _close as _close_rows
from test_gpu_qk_norm_rope import _pairsize

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF = torch.bfloat16


def test_rows_past_2_to_the_31_elements(gpu_lib):
    """One head of more than 2^31 elements.  At the usual decays 3000 tokens
    leave e^-100 or less of a state, so that the first and the last rows follow
    from the 4096 tokens at their end alone."""
    d, T, keep = 128, 4096, 1024
    L = 2 ** 31 // d + T + 37
    gen = torch.Generator(device=DEV).manual_seed(5)
    r = lambda: torch.randn((1, 1, L, d), generator=gen, device=DEV, dtype=BF)  # noqa: E731
    q, k, v, dO = r(), r().mul_(d ** -0.5), r(), r()
    g = torch.nn.functional.logsigmoid(torch.randn((1, 1, L), generator=gen, device=DEV) + 3)
    assert float(g[..., keep:T].sum()) < -100 and float(g[..., L - T:L - keep].sum()) < -100
    o, S = N.linear_chunk_fwd(q, k, v, g, out_dtype=BF)
    dq, dk, dv, dg, dS0 = N.linear_chunk_bwd(q, k, v, g, None, dO)
    torch.cuda.synchronize()
    for end in (slice(0, T), slice(L - T, L)):
        part = [to64(t[:, :, end]) for t in (q, k, v, g)]
        size = [np.abs(t) if i != 3 else t for i, t in enumerate(part)]
        do = to64(dO[:, :, end])
        oe, Se = linear_forward(*part)
        oa, Sa = linear_forward(*size)
        ge = linear_backward(*part, None, do)
        ga = linear_backward(*size, None, np.abs(do))
        # Where the end's own rows decide: behind 3072 tokens that are not the
        # tensor's first, in front of 3072 that are not its last.
        first = end.start == 0
        past = slice(0, keep) if first else slice(T - keep, T)
        cut = lambda t: t[:, :, end][:, :, past]  # noqa: E731
        _close(cut(o), oe[:, :, past], oa[:, :, past], BF, T, "o")
        for got, i, n in ((dq, 0, "dq"), (dk, 1, "dk"), (dv, 2, "dv")):
            _close(cut(got), ge[i][:, :, past], ga[i][:, :, past], BF, T, n)
        most = ga[3].max() * np.ones_like(ga[3][:, :, past])
        _close(cut(dg), ge[3][:, :, past], most, torch.float32, T, "dlog_decay", 2 * 256 + 3)
        if first:
            _close(dS0, ge[4], ga[4], torch.float32, T, "dS0")
        else:
            _close(S, Se, Sa, torch.float32, T, "S_final")


def test_most_heads(gpu_lib):
    x = _inputs(50, 257, 255, 1, 3, 64, 64, "bf16", True, "usual")
    g = _gpu(x)
    o, S = N.linear_chunk_fwd(g["q"], g["k"], g["v"], g["g"], g["S0"], out_dtype=BF)
    got = N.linear_chunk_bwd(g["q"], g["k"], g["v"], g["g"], g["S0"], g["dO"], g["dS"])
    S1 = g["S0"].clone()
    first = [g[n][:, :, 0].contiguous() for n in ("q", "k", "v", "g")]
    o1 = N.linear_decode_step(*first, S1)
    torch.cuda.synchronize()
    row = lambda t: None if t is None else t[[0, 130, 256]]  # noqa: E731
    x = {n: row(t) for n, t in x.items()}
    e, a = _np(x), _np(x, True)
    six = ("q", "k", "v", "g", "S0", "dO", "dS")
    want, size = linear_forward(*(e[n] for n in six[:5])), linear_forward(*(a[n] for n in six[:5]))
    _close(row(o), want[0], size[0], BF, 3, "o")
    _close(row(S), want[1], size[1], torch.float32, 3, "S_final")
    _close(row(o1), want[0][:, :, 0], size[0][:, :, 0], torch.float32, 3, "one token")
    want, size = linear_backward(*(e[n] for n in six)), linear_backward(*(a[n] for n in six))
    for i, n in enumerate(("dq", "dk", "dv")):
        _close(row(got[i]), want[i], size[i], BF, 3, n)
    _close(row(got[4]), want[4], size[4], torch.float32, 3, "dS0")
    most = size[3].max(-1, keepdims=True) * np.ones_like(size[3])
    _close(row(got[3]), want[3], most, torch.float32, 3, "dlog_decay", 4)


@pytest.mark.parametrize("L", [100, 700])
def test_decay_gradient_without_the_first_states(gpu_lib, L):
    """A start state whose own gradient is not asked for."""
    x = _inputs(51, 2, 2, 1, L, 64, 128, "bf16", True, "usual")
    g = _gpu(x)
    got = N.linear_chunk_bwd(g["q"], g["k"], g["v"], g["g"], g["S0"], g["dO"], g["dS"], want_dS0=False)
    assert got[4] is None
    e, a = _np(x), _np(x, True)
    names = ("q", "k", "v", "g", "S0", "dO", "dS")
    want, size = linear_backward(*(e[n] for n in names))[3], linear_backward(*(a[n] for n in names))[3]
    _close(got[3], want, size.max(-1, keepdims=True) * np.ones_like(size), torch.float32, L,
           "dlog_decay", 2 * L / 64 + 3)


def test_two_threads_on_two_streams(gpu_lib):
    xs = [_gpu(_inputs(52 + i, 2, 2, 2, 900, 128, 64, "bf16", True, "usual")) for i in range(2)]
    call = lambda x, s=None: (  # noqa: E731
        *N.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["S0"], stream=s),
        *N.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["S0"], x["dO"], x["dS"], stream=s))
    want = [call(x) for x in xs]
    torch.cuda.synchronize()
    bad = []

    def work(i):
        s = torch.cuda.Stream()
        for _ in range(20):
            got = call(xs[i], s)
            s.synchronize()
            bad.extend(n for n, (a, b) in enumerate(zip(want[i], got)) if not torch.equal(a, b))

    ts = [threading.Thread(target=work, args=(i,)) for i in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join()
    assert not bad


def test_two_graphs_on_one_workspace(gpu_lib):
    """Two captured calls that share the workspace that their caller gave, replayed
    in turn."""
    xs = [_gpu(_inputs(54 + i, 1, 2, 2, 700, 64, 64, "bf16", True, "usual")) for i in range(2)]
    n = N.linear_workspace_bytes(1, 4, 700, 64, 64, BF, 2, backward=True)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)
    call = lambda x, w: N.linear_chunk_bwd(  # noqa: E731
        x["q"], x["k"], x["v"], x["g"], x["S0"], x["dO"], x["dS"], workspace=w)
    want = [call(x, None) for x in xs]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for x in xs:
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            outs.append(call(x, ws))
    for _ in range(3):
        for gr in graphs:
            gr.replay()
        torch.cuda.synchronize()
        for w, o in zip(want, outs):
            for a, b in zip(w, o):
                assert torch.equal(a, b)
                b.zero_()


def test_second_derivatives_are_refused(gpu_lib):
    x = _gpu(_inputs(56, 1, 1, 1, 8, 64, 64, "f32", False, "usual"))
    q = x["q"].clone().requires_grad_()
    o, _ = N.linear_rule(q, x["k"], x["v"], x["g"])
    with pytest.raises(RuntimeError):
        torch.autograd.grad(torch.autograd.grad(o.sum(), q, create_graph=True)[0].sum(), q)
    y, _ = N.rotary_qk(q, x["k"], None, None)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(torch.autograd.grad(y.sum(), q, create_graph=True)[0].sum(), q)


def test_qk_rows_past_2_to_the_31_elements(gpu_lib):
    Hq, Hk, d, T = 31, 2, 128, 64
    L = 2 ** 31 // (Hq * d) + 2 * T + 5
    gen = torch.Generator(device=DEV).manual_seed(6)
    proj = torch.randn((1, L, Hq + Hk, d), generator=gen, device=DEV, dtype=BF)
    pos = torch.arange(L, device=DEV, dtype=torch.int32).view(1, L)
    inv = torch.from_numpy(10000.0 ** (-np.arange(64) / 64)).float().to(DEV)
    part = lambda t, i: t[:, :, :Hq].transpose(1, 2) if i == 0 else t[:, :, Hq:].transpose(1, 2)  # noqa: E731
    y = N.qk_norm_rope(part(proj, 0), part(proj, 1), pos, inv)
    dproj = torch.zeros_like(proj)
    N.qk_norm_rope_bwd(part(proj, 0), part(proj, 1), pos, inv, *y, dq_raw=part(dproj, 0),
                       dk_raw=part(dproj, 1))
    torch.cuda.synchronize()
    a = rotation_angles(to64(pos[:, -T:]), to64(inv))
    rel = (d / 8 + 24) * 2.0 ** -24
    for i, n in enumerate(("q", "k")):
        raw, dy = to64(part(proj, i)[:, :, -T:]), to64(y[i][:, :, -T:])
        flat = norm_rope(raw, None, np.zeros((1, T, 0)))
        _close_rows(y[i][:, :, -T:], norm_rope(raw, None, a), rel * _pairsize(flat, d // 2, False), n)
        dx, _ = norm_rope_backward(raw, None, a, dy)
        dn = _pairsize(dy.copy(), d // 2, False)
        r = 1 / np.sqrt((raw ** 2).mean(-1, keepdims=True) + 1e-6)
        xr = np.abs(raw) * r
        _close_rows(part(dproj, i)[:, :, -T:], dx, 2 * rel * r * (dn + xr * (xr * dn).mean(-1, keepdims=True)),
                    "d" + n)


def test_repeated_rows_are_read_in_place(gpu_lib):
    """Strides of 0: one row of q for all heads, one token of k for all tokens."""
    gen = torch.Generator(device=DEV).manual_seed(7)
    q = torch.randn((2, 1, 9, 64), generator=gen, device=DEV).expand(2, 4, 9, 64)
    k = torch.randn((2, 3, 1, 64), generator=gen, device=DEV).expand(2, 3, 9, 64)
    pos = torch.arange(18, device=DEV, dtype=torch.int32).view(2, 9)
    inv = torch.rand(32, generator=gen, device=DEV)
    got = N.qk_norm_rope(q, k, pos, inv)
    want = N.qk_norm_rope(q.contiguous(), k.contiguous(), pos, inv)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    got = N.qk_norm_rope_bwd(q, k, pos, inv, *want)
    want = N.qk_norm_rope_bwd(q.contiguous(), k.contiguous(), pos, inv, *want)
    for a, b in zip(got[:2], want[:2]):
        assert torch.equal(a, b)


def test_sums_over_shared_heads_in_more_than_one_round(gpu_lib):
    """More elements than the workgroups of the sums hold at once (fp32: what two
    heads leave is added exactly)."""
    L, d = 2 ** 18 + 70, 128
    assert 2 * L * d // 4 > 16384 * 1024
    gen = torch.Generator(device=DEV).manual_seed(8)
    r = lambda h, d=d: torch.randn((1, h, L, d), generator=gen, device=DEV)  # noqa: E731
    q, k, v, dO = r(1), r(1).mul_(d ** -0.5), r(2, 64), r(2, 64)
    g = torch.nn.functional.logsigmoid(torch.randn((1, 2, L), generator=gen, device=DEV) + 3)
    got = N.linear_chunk_bwd(q, k, v, g, None, dO)
    two = lambda t: t.expand(1, 2, L, d).contiguous()  # noqa: E731
    want = N.linear_chunk_bwd(two(q), two(k), v, g, None, dO)
    for a, b in zip(got[:2], want[:2]):
        assert torch.equal(a[:, 0], b[:, 0] + b[:, 1])
