"""The gated linear recurrence on the GPU against the fp64 oracle.

Bounds, element by element.  Every output is a sum of products; running the
oracle on absolute values gives A, the sum of the products' sizes.  Then
    |got - exact| <= u |exact| + E A
with u half a step of the output's type (``finfo.eps / 2``; 0 for fp32, whose
roundings are in E) and E the relative error of a term:
    n 2^-24   n = L + 512 fp32 roundings: one per token a value is carried over,
              the chunk's sums (64 + d) and the decay factors (a difference of
              fp64 sums rounded once to fp32, at most 150 in size where the
              factor is not zero, and the exponential);
    2^-16     where an fp32 operand enters a product as two bf16 pieces (what
              they leave of a value is at most 2^-17 of it, and both of a
              product's operands may be split), for bf16 outputs.
The decay's gradient is a difference of such sums along a head: its bound takes
the largest A of the head, three times per chunk it is carried over (a chunk's
x, y and D), at most 2 L / 64 + 3.
"""

import numpy as np
import pytest
import torch

from deltanet_delta_rule_chunk_amd import binding as N
from oracle import linear_backward, linear_decode_step, linear_forward
from parity import to64

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
T = {"bf16": torch.bfloat16, "f32": torch.float32}


def _gates(rng, kind, shape):
    if kind == "none":
        return None
    x = rng.standard_normal(shape)
    g = {"usual": -np.log1p(np.exp(-(x + 3))), "keep": np.zeros(shape), "slow": -1e-4 * np.abs(x),
         "strong": -8 - 4 * np.abs(x), "wiping": -np.log1p(np.exp(-(x + 3)))}[kind]
    if kind == "wiping":
        # wipes at single tokens, at both sides of a chunk's border and in a run
        for t in (0, 5, 63, 64, 65, 100, 101, 102, shape[-1] - 1):
            if t < shape[-1]:
                g[0, 0, t] = -np.inf
        g[..., shape[-1] // 2] = -np.inf
        g[-1, -1, :] = -300.0  # no wipe by value, one by effect
    return torch.from_numpy(g).float()


def _inputs(seed, B, Hqk, grp, L, dk, dv, dt, s0, gates):
    rng = np.random.default_rng(seed)
    H = Hqk * grp
    f = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(T[dt])  # noqa: E731
    x = dict(q=f(B, Hqk, L, dk), k=f(B, Hqk, L, dk) * dk ** -0.5, v=f(B, H, L, dv), dO=f(B, H, L, dv))
    x["g"] = _gates(rng, gates, (B, H, L))
    s = lambda: torch.from_numpy(rng.standard_normal((B, H, dk, dv))).float()  # noqa: E731
    x["S0"], x["dS"] = (s(), s()) if s0 else (None, None)
    return x


def _gpu(x):
    return {k: None if t is None else t.to(DEV) for k, t in x.items()}


def _np(x, size=False):
    """fp64 inputs; with ``size`` their absolute values (decays as they are)."""
    return {k: None if t is None else (np.abs(to64(t)) if size and k != "g" else to64(t))
            for k, t in x.items()}


def _close(got, exact, A, t, L, what, times=1.0):
    u = torch.finfo(t).eps / 2 if t == torch.bfloat16 else 0.0
    E = (L + 512) * 2.0 ** -24 + (2.0 ** -16 if t == torch.bfloat16 else 0.0)
    g = to64(got)
    assert np.isfinite(g).all(), what
    over = np.abs(g - exact) - (u * np.abs(exact) + times * E * A + 1e-37)
    assert (over <= 0).all(), f"{what}: {over.max():.3e} over the bound, {(over > 0).mean():.4f} of it"


CASES = [
    # B, Hqk, grp, L, dk, dv, dtype, state, gates
    (1, 1, 1, 1, 64, 64, "bf16", False, "usual"),
    (2, 3, 1, 1, 128, 128, "f32", True, "usual"),
    (1, 2, 1, 2, 64, 128, "bf16", True, "wiping"),
    (2, 1, 2, 63, 128, 64, "bf16", True, "usual"),
    (1, 2, 1, 64, 128, 128, "bf16", True, "none"),
    (1, 2, 1, 65, 64, 64, "f32", True, "wiping"),
    (1, 1, 3, 130, 64, 128, "bf16", False, "strong"),
    (1, 3, 1, 256, 128, 128, "bf16", True, "wiping"),
    (1, 2, 1, 257, 128, 64, "bf16", True, "usual"),     # a last chunk of one row
    (1, 1, 2, 257, 64, 128, "f32", False, "keep"),
    (2, 1, 3, 700, 64, 64, "bf16", True, "wiping"),
    (1, 1, 1, 1025, 128, 128, "bf16", True, "slow"),
    (1, 1, 2, 1090, 128, 128, "f32", True, "wiping"),
    (3, 2, 4, 333, 128, 64, "bf16", False, "none"),
    (1, 9, 1, 400, 64, 64, "bf16", True, "usual"),      # heads in no multiple of the XCDs
    (2, 101, 1, 300, 64, 64, "bf16", True, "wiping"),   # heads enough for one segment of several chunks
    (1, 60, 4, 193, 64, 64, "f32", True, "usual"),
]
IDS = ["-".join(map(str, c)) for c in CASES]


@pytest.mark.parametrize("case", CASES, ids=IDS)
@pytest.mark.parametrize("out", ["same", "other"])
def test_forward(gpu_lib, case, out):
    L, dt = case[3], case[6]
    x = _inputs(11, *case)
    t = T[dt] if out == "same" else T["f32" if dt == "bf16" else "bf16"]
    g = _gpu(x)
    o, S = N.linear_chunk_fwd(g["q"], g["k"], g["v"], g["g"], g["S0"], out_dtype=t)
    torch.cuda.synchronize()
    e, a = _np(x), _np(x, True)
    want = linear_forward(e["q"], e["k"], e["v"], e["g"], e["S0"])
    size = linear_forward(a["q"], a["k"], a["v"], a["g"], a["S0"])
    assert o.dtype == t
    _close(o, want[0], size[0], t, L, "o")
    _close(S, want[1], size[1], torch.float32, L, "S_final")


@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward(gpu_lib, case):
    L, dt = case[3], case[6]
    x = _inputs(12, *case)
    g = _gpu(x)
    got = N.linear_chunk_bwd(g["q"], g["k"], g["v"], g["g"], g["S0"], g["dO"], g["dS"])
    torch.cuda.synchronize()
    e, a = _np(x), _np(x, True)
    want = linear_backward(e["q"], e["k"], e["v"], e["g"], e["S0"], e["dO"], e["dS"])
    size = linear_backward(a["q"], a["k"], a["v"], a["g"], a["S0"], a["dO"], a["dS"])
    for i, name in enumerate(("dq", "dk", "dv")):
        assert got[i].dtype == T[dt]
        _close(got[i], want[i], size[i], T[dt], L, name)
    _close(got[4], want[4], size[4], torch.float32, L, "dS0")
    if x["g"] is None:
        assert got[3] is None
        return
    most = size[3].max(-1, keepdims=True) * np.ones_like(size[3])
    _close(got[3], want[3], most, torch.float32, L, "dlog_decay", 2 * L / 64 + 3)
    # The same in the mean: independent roundings add as the root of their
    # number, 2 L of them at most below 64^2.
    # (1e-37: what lies below fp32's smallest normal 2^-126 comes out as zero.)
    off = np.linalg.norm(to64(got[3]) - want[3])
    floor = 1e-37 * np.sqrt(size[3].size)
    assert off <= 64 * 2.0 ** -24 * np.linalg.norm(size[3]) + floor, off
    wiped = np.isinf(to64(x["g"]))
    assert (to64(got[3])[wiped] == 0).all()


def test_strong_decay_keeps_its_gradients_accuracy(gpu_lib):
    """At decays of e^-8 and below a token's own pair is thousands of times the
    decay's gradient: a gradient formed as a difference of both would be noise."""
    x = _inputs(13, 1, 2, 1, 640, 128, 128, "bf16", False, "strong")
    g = _gpu(x)
    got = N.linear_chunk_bwd(g["q"], g["k"], g["v"], g["g"], None, g["dO"])[3]
    e = _np(x)
    want = linear_backward(e["q"], e["k"], e["v"], e["g"], None, e["dO"])[3]
    rel = np.linalg.norm(to64(got) - want) / np.linalg.norm(want)
    # 64 rows' sums of fp32 products, and their chunk-to-chunk carries.
    assert rel < 640 * 2.0 ** -24, rel


def test_backward_against_differences_of_the_forward(gpu_lib):
    """A step along a random direction in fp32 inputs."""
    x = _gpu(_inputs(14, 1, 2, 2, 300, 64, 64, "f32", True, "usual"))
    gen = torch.Generator(device=DEV).manual_seed(3)
    names = ("q", "k", "v", "g", "S0")
    d = {n: torch.randn(x[n].shape, generator=gen, device=DEV) for n in names}

    def loss(h):
        y = {n: (x[n] + h * d[n]).contiguous() for n in names}
        o, S = N.linear_chunk_fwd(*(y[n] for n in names))
        return float((o.double() * x["dO"].double()).sum() + (S.double() * x["dS"].double()).sum())

    h = 2.0 ** -8
    num = (loss(h) - loss(-h)) / (2 * h)
    got = N.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["S0"], x["dO"], x["dS"])
    parts = [float((a.double() * d[n].double()).sum()) for a, n in zip(got, names)]
    size = np.sqrt(sum(p * p for p in parts))
    # third-order term h^2 and fp32 rounding of the two losses over 2 h
    assert abs(sum(parts) - num) <= 2e-3 * size, (parts, num)


def test_autograd(gpu_lib):
    x = _gpu(_inputs(15, 2, 2, 2, 130, 64, 128, "bf16", True, "usual"))
    leaves = [x[n].clone().requires_grad_() for n in ("q", "k", "v", "g", "S0")]
    o, S = N.linear_rule(*leaves)
    assert o.dtype == torch.bfloat16
    got = torch.autograd.grad([o, S], leaves, [x["dO"], x["dS"]])
    want = N.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["S0"], x["dO"], x["dS"])
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    # Broadcast gradients, an unused state, inputs that need none.
    q = x["q"].clone().requires_grad_()
    o, _ = N.linear_rule(q, x["k"], x["v"])
    o.sum().backward()
    want = N.linear_chunk_bwd(x["q"], x["k"], x["v"], None, None, torch.ones_like(x["v"]),
                              torch.zeros_like(x["S0"]))[0]
    assert torch.equal(q.grad, want)


DECODE = [(1, 1, 1, 64, 64, "bf16"), (3, 2, 3, 128, 64, "f32"), (2, 4, 1, 64, 128, "bf16"),
          (1, 32, 1, 128, 128, "bf16"), (40, 4, 4, 128, 128, "bf16"), (130, 8, 1, 64, 64, "f32")]


@pytest.mark.parametrize("B,Hqk,grp,dk,dv,dt", DECODE)
def test_decode_steps(gpu_lib, B, Hqk, grp, dk, dv, dt):
    rng = np.random.default_rng(16)
    H, t = Hqk * grp, T[dt]
    f = lambda *s: torch.from_numpy(rng.standard_normal(s)).to(t)  # noqa: E731
    S = torch.from_numpy(rng.standard_normal((B, H, dk, dv))).float()
    Sg, Se, Sa = S.to(DEV), to64(S), np.abs(to64(S))
    for step in range(3):
        q, k, v = f(B, Hqk, dk), f(B, Hqk, dk), f(B, H, dv)
        g = None if step == 2 else _gates(rng, "usual", (B, H))
        if step == 1:
            g[0, 0] = -float("inf")
        gg = None if g is None else g.to(DEV)
        o = N.linear_decode_step(q.to(DEV), k.to(DEV), v.to(DEV), gg, Sg, out_dtype=t)
        ge = None if g is None else to64(g)
        oe, Se = linear_decode_step(to64(q), to64(k), to64(v), ge, Se)
        oa, Sa = linear_decode_step(*(np.abs(to64(y)) for y in (q, k, v)), ge, Sa)
        # no operand is split here
        u = torch.finfo(t).eps / 2 if dt == "bf16" else 0.0
        assert (np.abs(to64(o) - oe) <= u * np.abs(oe) + (dk + 64) * 2.0 ** -24 * oa).all(), step
        assert (np.abs(to64(Sg) - Se) <= 16 * 2.0 ** -24 * Sa).all(), step


def test_decode_equals_a_forward_of_one_token(gpu_lib):
    x = _gpu(_inputs(17, 2, 2, 2, 1, 128, 128, "f32", True, "usual"))
    o, S = N.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["S0"])
    S2 = x["S0"].clone()
    o2 = N.linear_decode_step(x["q"][:, :, 0].contiguous(), x["k"][:, :, 0].contiguous(),
                              x["v"][:, :, 0].contiguous(), x["g"][:, :, 0].contiguous(), S2)
    scale = float(o.abs().max())
    assert float((o[:, :, 0] - o2).abs().max()) <= 512 * 2.0 ** -24 * scale
    assert float((S - S2).abs().max()) <= 8 * 2.0 ** -24 * float(S.abs().max())


def test_split_sequence_carries_its_state(gpu_lib):
    """Two calls with the state handed over are the one call, to rounding."""
    x = _gpu(_inputs(18, 1, 2, 1, 1000, 128, 128, "bf16", True, "usual"))
    whole, S = N.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["S0"])
    part = lambda a, b: [x[n][:, :, a:b].contiguous() for n in ("q", "k", "v", "g")]  # noqa: E731
    state = x["S0"].clone()
    outs = []
    for a, b in ((0, 333), (333, 334), (334, 1000)):
        o, _ = N.linear_chunk_fwd(*part(a, b), state, S_final=state)  # in place
        outs.append(o)
    both = torch.cat(outs, 2)
    assert float((both - whole).abs().max()) <= 1512 * 2.0 ** -24 * 16 * float(whole.abs().max())
    assert float((state - S).abs().max()) <= 1512 * 2.0 ** -24 * 16 * float(S.abs().max())


def test_no_tokens(gpu_lib):
    x = _gpu(_inputs(19, 1, 2, 1, 1, 64, 128, "bf16", True, "usual"))
    e = lambda n: x[n][:, :, :0].contiguous()  # noqa: E731
    o, S = N.linear_chunk_fwd(e("q"), e("k"), e("v"), e("g"), x["S0"])
    assert o.shape == (1, 2, 0, 128) and torch.equal(S, x["S0"])
    _, S = N.linear_chunk_fwd(e("q"), e("k"), e("v"), e("g"))
    assert not S.any()
    got = N.linear_chunk_bwd(e("q"), e("k"), e("v"), e("g"), x["S0"], e("dO"), x["dS"])
    assert torch.equal(got[4], x["dS"]) and got[0].numel() == 0


def test_same_bits_every_time(gpu_lib):
    x = _gpu(_inputs(20, 2, 2, 3, 1500, 128, 64, "bf16", True, "usual"))
    call = lambda: (*N.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["S0"]),  # noqa: E731
                    *N.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["S0"], x["dO"], x["dS"]))
    first = call()
    for _ in range(3):
        for a, b in zip(first, call()):
            assert torch.equal(a, b)


def test_packed_documents_do_not_see_each_other(gpu_lib):
    """Changing one document leaves the others' outputs and gradients bit for bit."""
    x = _gpu(_inputs(21, 1, 2, 1, 500, 64, 64, "bf16", False, "usual"))
    x["g"][..., 200] = -float("inf")
    x["g"][..., 301] = -float("inf")
    run = lambda: (*N.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"]),  # noqa: E731
                   *N.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], None, x["dO"]))
    a = run()
    for n in ("q", "k", "v", "dO"):
        x[n][:, :, 200:301] *= 3
    b = run()
    for i in (0, 2, 3, 4):  # o, dq, dk, dv
        assert torch.equal(a[i][:, :, :200], b[i][:, :, :200])
        assert torch.equal(a[i][:, :, 301:], b[i][:, :, 301:])
    assert torch.equal(a[1], b[1])
    assert not b[5][..., 200].any() and not b[5][..., 301].any()


def test_later_tokens_do_not_reach_earlier_ones(gpu_lib):
    x = _gpu(_inputs(22, 1, 1, 1, 200, 64, 64, "bf16", False, "usual"))
    a, _ = N.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"])
    for n in ("q", "k", "v"):
        x[n][:, :, 70:] = 7
    b, _ = N.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"])
    assert torch.equal(a[:, :, :70], b[:, :, :70])


def test_stream_workspace_and_library_scratch(gpu_lib):
    """Another stream; a given workspace full of NaN; the library's own
    stream-ordered allocation (null workspace) through the C ABI."""
    x = _gpu(_inputs(23, 2, 2, 1, 900, 64, 128, "bf16", True, "usual"))
    ref = N.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["S0"])
    refb = N.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["S0"], x["dO"], x["dS"])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = N.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["S0"], stream=side)
    outb = N.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["S0"], x["dO"], x["dS"], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip((*ref, *refb), (*out, *outb)):
        assert torch.equal(a, b)
    for bwd in (False, True):
        n = N.linear_workspace_bytes(2, 2, 900, 64, 128, torch.bfloat16, backward=bwd)
        assert n > 0 and n % 4 == 0
        ws = torch.full((n // 4,), float("nan"), device=DEV)
        if bwd:
            got = N.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["S0"], x["dO"], x["dS"],
                                     workspace=ws)
        else:
            got = N.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["S0"], workspace=ws)
        for a, b in zip(refb if bwd else ref, got):
            assert torch.equal(a, b)
    o, S = torch.empty_like(ref[0]), torch.empty_like(ref[1])
    st = gpu_lib.deltanet_linear_chunk_fwd(
        x["q"].data_ptr(), x["k"].data_ptr(), x["v"].data_ptr(), x["g"].data_ptr(),
        x["S0"].data_ptr(), o.data_ptr(), S.data_ptr(), 2, 2, 2, 900, 64, 128, 1, 0, None, 0,
        torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    assert torch.equal(o, ref[0]) and torch.equal(S, ref[1])


def test_captured_and_replayed(gpu_lib):
    """Forward, backward and a decode step in a graph, replayed on new inputs
    with eager calls of the same operators between the replays."""
    x = _gpu(_inputs(24, 1, 2, 2, 600, 64, 64, "bf16", True, "usual"))
    names = ("q", "k", "v", "g")
    S = x["S0"].clone()

    def call():
        out = (*N.linear_chunk_fwd(*(x[n] for n in names), x["S0"]),
               *N.linear_chunk_bwd(*(x[n] for n in names), x["S0"], x["dO"], x["dS"]))
        S.copy_(x["S0"])
        row = [x[n][:, :, 3].contiguous() for n in names]
        return (*out, N.linear_decode_step(*row, S), S)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        static = call()
    for i in range(4):
        new = _gpu(_inputs(30 + i, 1, 2, 2, 600, 64, 64, "bf16", True, "usual"))
        for n in x:
            x[n].copy_(new[n])
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in static]
        for a, b in zip(kept, call()):
            assert torch.equal(a, b), i


def test_rows_behind_the_last_are_left_alone(gpu_lib):
    """Outputs sit between guard elements in one allocation."""
    x = _gpu(_inputs(25, 1, 1, 1, 70, 64, 64, "bf16", True, "usual"))
    n = 70 * 64
    buf = torch.full((n + 512,), 5.0, device=DEV)
    o = buf[256:256 + n].view(1, 1, 70, 64)
    N.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["S0"], o=o)
    torch.cuda.synchronize()
    assert (buf[:256] == 5).all() and (buf[256 + n:] == 5).all()


def test_non_finite_rows_stay_in_their_chunk_and_after(gpu_lib):
    x = _gpu(_inputs(26, 1, 1, 1, 300, 64, 64, "bf16", False, "usual"))
    ref, _ = N.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"])
    x["v"][0, 0, 130] = float("inf")
    x["q"][0, 0, 150] = float("nan")
    o, S = N.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"])
    assert torch.equal(o[:, :, :128], ref[:, :, :128])
    assert not torch.isfinite(o[:, :, 130:]).any() and not torch.isfinite(S).any()


@pytest.mark.parametrize("L,dt,grp", [(1, "bf16", 1), (64, "f32", 1), (200, "bf16", 2), (900, "bf16", 1), (900, "f32", 3)])
@pytest.mark.parametrize("junk", [float("nan"), float("inf")])
def test_a_wipe_drops_any_state(gpu_lib, L, dt, grp, junk):
    """A wipe at a sequence's first token: what the state's buffer held, memory
    never written among it, does not show, in any output or gradient."""
    x = _gpu(_inputs(29, 1, 2, grp, L, 128, 64, dt, True, "usual"))
    x["g"][..., 0] = -float("inf")

    def call(S0):
        S = S0.clone()
        row = [x[n][:, :, 0].contiguous() for n in ("q", "k", "v", "g")]
        return (*N.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], S0),
                *N.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], S0, x["dO"], x["dS"]),
                N.linear_decode_step(*row, S), S)

    want, got = call(torch.zeros_like(x["S0"])), call(torch.full_like(x["S0"], junk))
    for a, b in zip(want, got):
        assert torch.isfinite(b).all() and torch.equal(a, b)


def test_profile_slots(gpu_lib):
    x = _gpu(_inputs(27, 1, 2, 1, 600, 64, 64, "bf16", True, "usual"))
    N.profile_start()
    N.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"])
    N.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], None, x["dO"])
    got = N.profile_stop()
    # forward: segment sums, their combination, outputs; backward: the same
    # two, the walks and the decay's gradient
    assert got["linear_out"][1] == 1 and got["linear_state"][1] == 4 and got["linear_bwd"][1] == 2
    assert all(ms > 0 for ms, _ in got.values())


def test_binding_refusals(gpu_lib):
    x = _gpu(_inputs(28, 1, 2, 1, 8, 64, 64, "bf16", True, "usual"))
    q, k, v, g = (x[n] for n in ("q", "k", "v", "g"))
    with pytest.raises(ValueError, match="contiguous"):
        N.linear_chunk_fwd(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, g)
    with pytest.raises(ValueError, match="log_decay"):
        N.linear_chunk_fwd(q, k, v, g[..., :4])
    with pytest.raises(ValueError, match="dtype"):
        N.linear_chunk_fwd(q, k, v.float(), g)
    with pytest.raises(ValueError, match="dO"):
        N.linear_chunk_bwd(q, k, v, g, None, x["dO"].float())
    with pytest.raises(N.DeltaNetError):
        N.linear_chunk_fwd(q, k, torch.cat([v, v[:, :1]], 1), torch.zeros(1, 3, 8, device=DEV))
    with pytest.raises(TypeError):
        N.linear_chunk_fwd(q.half(), k.half(), v.half(), g)
    with pytest.raises(N.DeltaNetError):
        y = torch.zeros(1, 2, 2000, 64, dtype=torch.bfloat16, device=DEV)
        N.linear_chunk_fwd(y, y.clone(), y.clone(), None,
                           workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
