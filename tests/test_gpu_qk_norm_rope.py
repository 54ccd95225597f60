"""The q / k norm with rotation on the GPU against the fp64 oracle.

Bounds.  A normed element is x r w: r carries the fp32 sum of d squares (each
partial sum rounds once: at most d / 8 + 8 of them on a path, relative to a sum
of positive terms), a square root, a division and the mean's product, and x r w
two products: (d / 8 + 16) 2^-24 of its size.  A turned element is a sum of two
products with cos and sin, each within 4 x 2^-24 of its fp32 angle's, whose own
error is half a step of a number below pi (2^-23): 8 x 2^-24 of |a| + |b|.
Outputs round to their type (``finfo.eps / 2``).
"""

import numpy as np
import pytest
import torch

from deltanet_delta_rule_chunk_amd import binding as N
from oracle import norm_rope, norm_rope_backward, rotate, rotation_angles
from parity import to64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
T = {"bf16": torch.bfloat16, "f32": torch.float32}

CASES = [
    # B, Hq, Hk, L, d, d_rot, sections, interleaved, norm, weights, dtype
    (1, 1, 1, 1, 128, 128, None, False, True, True, "bf16"),
    (2, 4, 2, 33, 128, 128, None, False, True, True, "bf16"),
    (2, 4, 2, 33, 128, 128, None, True, True, True, "f32"),
    (1, 3, 1, 100, 64, 64, [8, 12, 12], False, True, True, "bf16"),
    (3, 5, 0, 7, 64, 48, [10, 14], True, True, False, "f32"),
    (1, 2, 7, 65, 128, 64, None, False, True, True, "f32"),
    (2, 2, 1, 19, 128, 0, None, False, True, True, "bf16"),
    (1, 2, 2, 40, 64, 64, None, False, False, True, "bf16"),
    (1, 2, 2, 40, 128, 104, [0, 50, 1, 1], True, False, False, "f32"),
    (5, 9, 3, 129, 64, 16, None, False, True, True, "bf16"),
    (1, 32, 8, 2500, 64, 64, None, False, True, True, "bf16"),
    (1, 41, 23, 2100, 64, 32, None, True, True, True, "bf16"),  # several token blocks per workgroup
]


def _inputs(seed, B, Hq, Hk, L, d, d_rot, sections, interleaved, norm, weights, dt):
    rng = np.random.default_rng(seed)
    t = T[dt]
    f = lambda *s: torch.from_numpy(rng.standard_normal(s))  # noqa: E731
    x = {}
    proj = f(B, L, Hq + 2 * Hk + 1, d).to(t).to(DEV)
    x["q_raw"] = proj[:, :, :Hq].transpose(1, 2)
    x["k_raw"] = proj[:, :, Hq:Hq + Hk].transpose(1, 2)
    x["dq_hat"], x["dk_hat"] = f(B, Hq, L, d).to(t).to(DEV), f(B, Hk, L, d).to(t).to(DEV)
    x["positions"] = x["inv_freq"] = None
    axes = 1 if sections is None else len(sections)
    if d_rot:
        p = rng.integers(-1000, 1 << 21, (axes, B, L))
        p.flat[0] = 2 ** 31 - 1
        p.flat[-1] = 0
        x["positions"] = torch.from_numpy(p.astype(np.int32)).to(DEV)
        x["inv_freq"] = torch.from_numpy(10000.0 ** (-np.arange(d_rot // 2) / (d_rot // 2))).float().to(DEV)
    how = dict(sections=sections, eps=1e-6, norm=norm, interleaved=interleaved)
    for n in ("q_weight", "k_weight"):
        how[n] = (1 + 0.3 * f(d)).float().to(DEV) if weights else None
    return x, how


def _angles(x, how, L, B):
    if x["inv_freq"] is None:
        return np.zeros((B, L, 0))
    return rotation_angles(to64(x["positions"]), to64(x["inv_freq"]), how["sections"])


def _np(t):
    return None if t is None else to64(t)


def _pairsize(y, n, interleaved):
    """|a| + |b| of each element's pair, |a| for elements that do not turn."""
    s = np.abs(y)
    if n:
        ia, ib = ((slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved
                  else (slice(0, n), slice(n, 2 * n)))
        both = s[..., ia] + s[..., ib]
        s[..., ia], s[..., ib] = both, both
    return s


def _close(got, exact, tol, what):
    g = to64(got)
    u = torch.finfo(got.dtype).eps / 2 if got.dtype == torch.bfloat16 else 2.0 ** -24
    over = np.abs(g - exact) - (u * np.abs(exact) + tol + 1e-37)
    assert (over <= 0).all(), f"{what}: {over.max():.3e} over the bound, {(over > 0).mean():.4f} of it"


@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c)) for c in CASES])
def test_forward_and_backward(gpu_lib, case):
    B, Hq, Hk, L, d, d_rot = case[:6]
    x, how = _inputs(1, *case)
    y = N.qk_norm_rope(x["q_raw"], x["k_raw"], x["positions"], x["inv_freq"], **how)
    grads = N.qk_norm_rope_bwd(x["q_raw"], x["k_raw"], x["positions"], x["inv_freq"], x["dq_hat"],
                               x["dk_hat"], **how)
    torch.cuda.synchronize()
    a = _angles(x, how, L, B)
    n, inter, norm = d_rot // 2, how["interleaved"], how["norm"]
    rel = (d / 8 + 24) * 2.0 ** -24
    for i, name in enumerate(("q", "k")):
        if y[i].numel() == 0:
            continue
        raw, w = _np(x[name + "_raw"]), _np(how[name + "_weight"])
        want = norm_rope(raw, w, a, 1e-6, norm, inter)
        flat = norm_rope(raw, w, np.zeros((B, L, 0)), 1e-6, norm, inter)
        assert y[i].is_contiguous()
        _close(y[i], want, rel * _pairsize(flat, n, inter), name + "_hat")
        dy = _np(x["d" + name + "_hat"])
        dx, dw = norm_rope_backward(raw, w, a, dy, 1e-6, norm, inter)
        # dn and what multiplies it, in size; the mean's product adds the row's.
        dn = _pairsize(dy.copy(), n, inter) * (1 if w is None else np.abs(w))
        r = 1 / np.sqrt((raw * raw).mean(-1, keepdims=True) + 1e-6) if norm else np.ones(raw.shape[:-1] + (1,))
        xh = np.abs(raw) * r
        size = r * (dn + xh * (xh * dn).mean(-1, keepdims=True)) if norm else dn
        _close(grads[i], dx, 3 * rel * size, "d" + name + "_raw")
        if w is None:
            assert grads[2 + i] is None
            continue
        # fp32 sums along a lane's rows, a workgroup's and all of them in fp64:
        # at most the rows of one lane plus 64 roundings of the running sum.
        rows = raw.shape[1] * (-(-B * L // 16) // 1024 + 1) + 64
        dw_size = (_pairsize(dy.copy(), n, inter) * xh).sum((0, 1, 2))
        _close(grads[2 + i], dw, (3 * rel + rows * 2.0 ** -24) * dw_size, "d" + name + "_weight")


def test_far_positions_are_exact_angles(gpu_lib):
    """A position of millions times the fastest frequency, in fp32: the angle's
    error is that of the turn's rest, not of its millions of radians."""
    L = 64
    p = torch.arange(2 ** 31 - L, 2 ** 31, device=DEV).to(torch.int32)[None].contiguous()
    f = torch.linspace(0.9, 1.0, 32, device=DEV)
    x = torch.ones(1, 1, L, 64, device=DEV)
    y, _ = N.qk_norm_rope(x, x[:, :0], p, f, norm=False)
    want = rotate(to64(x), rotation_angles(to64(p), to64(f)))
    # fp64 turns: 2^31 / (2 pi) x 2^-52 turns off at most, besides fp32's 16 x 2^-24.
    tol = 2 * (2.0 ** 31 * 2.0 ** -52 + 16 * 2.0 ** -24)
    assert np.abs(to64(y) - want).max() <= tol


def test_layouts_agree_bit_for_bit(gpu_lib):
    """The fused projection's rows, dense copies, repeated (stride 0) rows."""
    x, how = _inputs(2, 2, 4, 2, 37, 128, 96, None, False, True, True, "bf16")
    call = lambda q, k: N.qk_norm_rope(q, k, x["positions"], x["inv_freq"], **how)  # noqa: E731
    ref = call(x["q_raw"], x["k_raw"])
    assert not x["q_raw"].is_contiguous()
    for a, b in zip(ref, call(x["q_raw"].contiguous(), x["k_raw"].contiguous())):
        assert torch.equal(a, b)
    one = x["k_raw"][:, :1].contiguous()
    for a, b in zip(call(x["q_raw"], one.expand(2, 2, 37, 128)),
                    call(x["q_raw"], one.repeat(1, 2, 1, 1))):
        assert torch.equal(a, b)


def test_gradient_into_the_fused_projection(gpu_lib):
    """dq_raw and dk_raw as parts of one buffer, whose other rows stay."""
    x, how = _inputs(3, 2, 4, 2, 21, 64, 64, None, False, True, True, "bf16")
    args = (x["q_raw"], x["k_raw"], x["positions"], x["inv_freq"], x["dq_hat"], x["dk_hat"])
    ref = N.qk_norm_rope_bwd(*args, **how)
    buf = torch.full((2, 21, 8, 64), 3.0, dtype=torch.bfloat16, device=DEV)
    got = N.qk_norm_rope_bwd(*args, **how, dq_raw=buf[:, :, :4].transpose(1, 2),
                             dk_raw=buf[:, :, 4:6].transpose(1, 2))
    for a, b in zip(ref, got):
        assert torch.equal(a, b)
    assert (buf[:, :, 6:] == 3).all()


def test_autograd_through_a_fused_projection(gpu_lib):
    x, how = _inputs(4, 1, 4, 2, 50, 64, 64, [16, 8, 8], False, True, True, "f32")
    proj = torch.randn(1, 50, 8, 64, device=DEV, requires_grad=True)
    qw = how["q_weight"].requires_grad_()
    q, k = N.rotary_qk(proj[:, :, :4].transpose(1, 2), proj[:, :, 4:6].transpose(1, 2),
                       x["positions"], x["inv_freq"], **how)
    dp, dw = torch.autograd.grad([q, k], [proj, qw], [x["dq_hat"], x["dk_hat"]])
    want = N.qk_norm_rope_bwd(proj[:, :, :4].transpose(1, 2), proj[:, :, 4:6].transpose(1, 2),
                              x["positions"], x["inv_freq"], x["dq_hat"], x["dk_hat"], **how)
    assert torch.equal(dp[:, :, :4].transpose(1, 2), want[0])
    assert torch.equal(dp[:, :, 4:6].transpose(1, 2), want[1])
    assert not dp[:, :, 6:].any() and torch.equal(dw, want[2])


def test_gradient_against_differences(gpu_lib):
    x, how = _inputs(5, 1, 2, 1, 30, 64, 64, None, True, True, True, "f32")
    d = torch.randn(x["q_raw"].shape, device=DEV, generator=torch.Generator(DEV).manual_seed(1))

    def loss(h):
        y, _ = N.qk_norm_rope(x["q_raw"] + h * d, x["k_raw"], x["positions"], x["inv_freq"], **how)
        return float((y.double() * x["dq_hat"].double()).sum())

    h = 2.0 ** -7
    num = (loss(h) - loss(-h)) / (2 * h)
    got = N.qk_norm_rope_bwd(x["q_raw"], x["k_raw"], x["positions"], x["inv_freq"], x["dq_hat"],
                             x["dk_hat"], **how)[0]
    part = (got.double() * d.double())
    assert abs(float(part.sum()) - num) <= 2e-3 * float(part.square().sum().sqrt())


def test_zero_and_huge_rows(gpu_lib):
    x = torch.zeros(1, 1, 3, 64, device=DEV)
    x[0, 0, 1] = 1e20
    x[0, 0, 2] = 1e-20
    y, _ = N.qk_norm_rope(x, x[:, :0], None, None)
    assert not y[0, 0, 0].any() and not y[0, 0, 1].any()  # zeros; the sum of squares overflows
    np.testing.assert_allclose(to64(y[0, 0, 2]), 1e-17, rtol=1e-6)


def test_bits_streams_and_graphs(gpu_lib):
    x, how = _inputs(6, 2, 3, 3, 77, 128, 128, [20, 20, 24], False, True, True, "bf16")

    def call(**kw):
        lead = (x["q_raw"], x["k_raw"], x["positions"], x["inv_freq"])
        return (*N.qk_norm_rope(*lead, **how, **kw),
                *N.qk_norm_rope_bwd(*lead, x["dq_hat"], x["dk_hat"], **how, **kw))

    ref = call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = call(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(ref, other):
        assert torch.equal(a, b)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = call()
    for i in range(4):
        new, _ = _inputs(40 + i, 2, 3, 3, 77, 128, 128, [20, 20, 24], False, True, True, "bf16")
        for n in x:
            x[n].copy_(new[n])
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in static]
        for a, b in zip(kept, call()):
            assert torch.equal(a, b), i


def test_no_tokens(gpu_lib):
    x, how = _inputs(7, 1, 2, 1, 4, 64, 64, None, False, True, True, "bf16")
    q, k = x["q_raw"][:, :, :0], x["k_raw"][:, :, :0]
    p = x["positions"][:, :, :0].contiguous()
    y = N.qk_norm_rope(q, k, p, x["inv_freq"], **how)
    assert y[0].shape == (1, 2, 0, 64)
    g = N.qk_norm_rope_bwd(q, k, p, x["inv_freq"], y[0], y[1], **how)
    assert not g[2].any() and not g[3].any()


def test_binding_refusals(gpu_lib):
    x, how = _inputs(8, 1, 2, 1, 4, 64, 64, None, False, True, True, "bf16")
    call = lambda **kw: N.qk_norm_rope(*({**x, **kw}[n] for n in  # noqa: E731
                                         ("q_raw", "k_raw", "positions", "inv_freq")), **how)
    with pytest.raises(ValueError, match="int32"):
        call(positions=x["positions"].long())
    with pytest.raises(ValueError, match="positions"):
        call(positions=None)
    with pytest.raises(ValueError, match="sections"):
        call(positions=x["positions"].expand(2, 1, 4).contiguous())
    with pytest.raises(ValueError, match="last dimension"):
        call(q_raw=x["q_raw"].transpose(2, 3).contiguous().transpose(2, 3))
    with pytest.raises(ValueError, match="q_weight"):
        N.qk_norm_rope(x["q_raw"], x["k_raw"], None, None, q_weight=torch.ones(32, device=DEV))
    with pytest.raises(N.DeltaNetError):
        N.qk_norm_rope(x["q_raw"], x["k_raw"], x["positions"], x["inv_freq"], sections=[31])
    with pytest.raises(N.DeltaNetError):
        N.qk_norm_rope(x["q_raw"], x["k_raw"], x["positions"], x["inv_freq"][:10].contiguous())
