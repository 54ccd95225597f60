"""The selective scan against the fp64 one, forward, backward and token by token.

Bounds, in fp32 roundings of the terms' magnitudes.  A step dt = softplus(raw + bias) is
off by (2.5 |raw + bias| + 6) of itself, |raw + bias| < 10 here: 31.  A decay
e^(dt A) over many tokens is off by (1 of exp2 and 1 of the product) per token and by 33 X
e^-X <= 12 through the steps, X the exponent.  A state adds a product and a sum
per token.  So 4 per token and 64 cover states, outputs and their sums over 32 states;
gradients pass the same a second time, and sums over channels and tokens one rounding
each of at most 16 + 64 + L of their terms: 8 per token and 256.
"""

import numpy as np
import pytest
import torch

from deltanet_delta_rule_chunk_amd import binding as N
from oracle import scan_backward, scan_forward, spans_of
from ssm_cases import DEV, PACKED, close, cu_of, f64, gpu, normal, scan_inputs

pytestmark = pytest.mark.gpu
IN = ("u", "dt", "A", "B", "C")
HOW = ("D", "z", "dt_bias", "h0")
NAMES = ("du", "ddt", "dA", "dB", "dC", "dD", "dz", "ddt_bias", "dh0")


def _how(x):
    return {n: x[n] for n in HOW}


def _forward(x, **more):
    return N.selective_scan_fwd(*(x[n] for n in IN), **_how(x), **more)


def _backward(x, **more):
    return N.selective_scan_bwd(*(x[n] for n in IN), x["dy"], x["dhT"], **_how(x), **more)


def _check(x, g, cuts=None, softplus=True):
    B, L, _ = x["u"].shape
    e, spans, cu = {k: f64(v) for k, v in x.items()}, spans_of(B, L, cuts), cu_of(cuts)
    y, hT = _forward(g, softplus=softplus, cu_seqlens=cu)
    how = dict(**_how(e), softplus=softplus)
    args = [e[n] for n in IN]
    want, size = scan_forward(*args, spans, **how), scan_forward(*args, spans, **how, size=True)
    longest = max((hi - lo for _, lo, hi in spans), default=0)
    close(y, want[0], size[0], 4 * longest + 64, "y")
    close(hT, want[1], size[1], 4 * longest + 64, "hT")
    got = _backward(g, softplus=softplus, cu_seqlens=cu)
    how = (*args, e["dy"], e["dhT"], spans)
    more = dict(**_how(e), softplus=softplus)
    want, size = scan_backward(*how, **more), scan_backward(*how, **more, size=True)
    for i, n in enumerate(NAMES):
        if got[i] is not None:
            close(got[i], want[i], size[i], 8 * longest + 256 + (L if i in (2, 5, 7) else 0), n)
    for i, n in ((5, "D"), (6, "z"), (7, "dt_bias")):
        assert (got[i] is None) == (x[n] is None)
    outside = np.ones((B, L), bool)
    for row, lo, hi in spans:
        outside[row, lo:hi] = False
    outside = torch.from_numpy(outside)
    for t in (y, got[0], got[1], got[3], got[4], got[6]):
        assert t is None or not t.cpu()[outside].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S", [8, 16, 32])
@pytest.mark.parametrize("B,L,D", [(1, 1, 8), (3, 2, 72), (2, 16, 64), (2, 31, 136), (1, 64, 8), (2, 65, 24), (1, 300, 64)])
def test_batch(gpu_lib, dtype, S, B, L, D):
    x = scan_inputs(L + S, B, L, D, S, dtype, B)
    _check(x, gpu(x))


@pytest.mark.parametrize("B,L,D", [(1, 80, 256), (1, 81, 256), (2, 33, 264), (1, 400, 1024), (1, 700, 1024), (5, 300, 1024), (9, 130, 1024), (33, 40, 1024)])
def test_lengths_of_segments(gpu_lib, B, L, D):
    """Around the rules that choose whether, and into pieces of how many tokens, sequences are cut."""
    x = scan_inputs(L, B, L, D, 8, "f32", B)
    _check(x, gpu(x))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("where", PACKED)
@pytest.mark.parametrize("S", [8, 16])
def test_packed(gpu_lib, dtype, where, S):
    L, cuts = PACKED[where]
    x = scan_inputs(L + S, 1, L, 72, S, dtype, len(cuts) - 1)
    _check(x, gpu(x), cuts)


@pytest.mark.parametrize("state,gate,skip,bias,softplus", [
    (False, True, True, True, True), (True, False, True, True, True), (True, True, False, False, True),
    (False, False, False, False, True), (True, False, False, True, False)])
def test_forms(gpu_lib, state, gate, skip, bias, softplus):
    for cuts in (None, [0, 3, 3, 80, 100]):
        x = scan_inputs(4, 1, 101, 24, 16, "bf16", 1 if cuts is None else 4, state, gate, skip, bias)
        if not softplus:
            x["dt"], x["dt_bias"] = x["dt"].abs() * 0.05, x["dt_bias"].abs() * 0.01
        _check(x, gpu(x), cuts, softplus)


def test_enough_sequences_for_one_walk(gpu_lib):
    """514 workgroups without a cut, sequences of several tiles."""
    x = scan_inputs(5, 257, 70, 72, 16, "f32", 257)
    _check(x, gpu(x))


def test_many_packed_sequences(gpu_lib):
    """More than one pass of the segments' table, lengths from 0 to 40."""
    rng = np.random.default_rng(0)
    cuts = np.concatenate([[2], 2 + np.cumsum(rng.integers(0, 41, 300) * (rng.random(300) < 0.5))]).tolist()
    x = scan_inputs(6, 1, cuts[-1] + 5, 16, 8, "f32", 300)
    _check(x, gpu(x), cuts)


def test_rows_out_of_projections(gpu_lib):
    x = scan_inputs(7, 2, 37, 64, 16, "bf16", 2)
    g = gpu(x)
    wide = torch.randn((2, 37, 256), device=DEV).to(torch.bfloat16)
    few = torch.randn((2, 37, 48), device=DEV).to(torch.bfloat16)
    wide[..., 64:128], wide[..., 192:] = g["u"], g["z"]
    few[..., 16:32], few[..., 32:] = g["B"], g["C"]
    g["u"], g["z"], g["B"], g["C"] = wide[..., 64:128], wide[..., 192:], few[..., 16:32], few[..., 32:]
    _check(x, g)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S", [8, 16, 32])
@pytest.mark.parametrize("gate", [True, False])
def test_tokens_one_by_one(gpu_lib, dtype, S, gate):
    x = scan_inputs(8, 5, 6, 72, S, dtype, 5, gate=gate)
    g = gpu(x)
    e, spans = {k: f64(v) for k, v in x.items()}, spans_of(5, 6)
    h, rows = g["h0"].clone(), []
    for t in range(6):
        rows.append(N.selective_scan_step(g["u"][:, t], g["dt"][:, t], g["A"], g["B"][:, t], g["C"][:, t], h, D=g["D"],
                                          z=g["z"][:, t] if gate else None, dt_bias=g["dt_bias"]))
    args = [e[n] for n in IN]
    want, size = scan_forward(*args, spans, **_how(e)), scan_forward(*args, spans, **_how(e), size=True)
    close(torch.stack(rows, 1), want[0], size[0], 4 * 6 + 64, "y")
    close(h, want[1], size[1], 4 * 6 + 64, "h")


@pytest.mark.parametrize("L", [40, 300])
def test_state_in_place(gpu_lib, L):
    x = gpu(scan_inputs(9, 2, L, 72, 16, "bf16", 2))
    y, hT = _forward(x)
    h = x["h0"].clone()
    y1, h1 = _forward(dict(x, h0=h), hT=h)
    assert h1 is h and torch.equal(h, hT) and torch.equal(y, y1)
    assert _forward(x, want_state=False)[1] is None


def test_extreme_steps(gpu_lib):
    """raw from far below (a step of nothing) to far above (the state is gone), rates of
    zero among A: all finite, and as the formula says."""
    x = scan_inputs(10, 1, 40, 64, 16, "f32", 1, bias=False)
    x["dt"] = torch.linspace(-9.5, 9.5, 40 * 64).reshape(1, 40, 64)
    x["A"][::3, ::2] = 0.0
    _check(x, gpu(x))
    x["dt"][:, 5] = -200.0   # no step at all: the state stays
    x["dt"][:, 9] = 3000.0   # the decay is 0 wherever A is not
    g = gpu(x)
    y, hT = _forward(g)
    assert torch.isfinite(y).all() and torch.isfinite(hT).all()
    e, spans = {k: f64(v) for k, v in x.items()}, spans_of(1, 40)
    want = scan_forward(*(e[n] for n in IN), spans, **_how(e))
    size = scan_forward(*(e[n] for n in IN), spans, **_how(e), size=True)
    # (2.5 roundings of an exponent per 2^-24: those of 3000 leave nothing of the decay either way.)
    close(hT, want[1], size[1], 4 * 40 + 64, "hT")
    assert all(torch.isfinite(t).all() for t in _backward(g) if t is not None)


def test_what_is_not_finite_stays_in_its_sequence_and_channel(gpu_lib):
    cuts = [0, 70, 150, 290]
    x = gpu(scan_inputs(11, 1, 300, 64, 16, "bf16", 3))
    cu = cu_of(cuts)
    want = (*_forward(x, cu_seqlens=cu), *_backward(x, cu_seqlens=cu))
    bad = {k: None if v is None else v.clone() for k, v in x.items()}
    for n in ("u", "dt", "B", "C", "z", "dy"):
        bad[n][:, 70:150] = float("nan")
        bad[n][:, 290:] = float("inf")
    for n in ("h0", "dhT"):
        bad[n][1] = float("nan")
    got = (*_forward(bad, cu_seqlens=cu), *_backward(bad, cu_seqlens=cu))
    keep = [i for i in range(290) if not 70 <= i < 150]
    for i in (0, 2, 3, 5, 6, 8):   # y, du, ddt, dB, dC, dz
        assert torch.equal(got[i][:, keep], want[i][:, keep]) and not got[i][:, 290:].any(), i
    for i in (1, 10):
        assert torch.equal(got[i][[0, 2]], want[i][[0, 2]])
    # One channel's input: the other channels.
    bad = {k: None if v is None else v.clone() for k, v in x.items()}
    bad["u"][:, 100, 5] = float("inf")
    got = (*_forward(bad, cu_seqlens=cu), *_backward(bad, cu_seqlens=cu))
    others = [d for d in range(64) if d != 5]
    for i in (0, 2, 3, 8):
        assert torch.equal(got[i][..., others], want[i][..., others]), i
    assert torch.equal(got[4][others], want[4][others])


def test_cuts_that_fall_or_leave_the_rows_stay_in_bounds(gpu_lib):
    x = gpu(scan_inputs(12, 1, 140, 64, 16, "bf16", 4))
    for cuts in ([0, 100, 10, 150, 140], [-7, 5, 5, 2 ** 31 - 1, 3], [150, 160, 170, 180, 190]):
        out = (*_forward(x, cu_seqlens=cu_of(cuts)), *_backward(x, cu_seqlens=cu_of(cuts)))
        torch.cuda.synchronize()
        assert all(torch.isfinite(t.float()).all() for t in out)


def test_no_tokens(gpu_lib):
    x = gpu(scan_inputs(13, 2, 0, 64, 16, "bf16", 2))
    y, hT = _forward(x)
    assert y.shape == (2, 0, 64) and torch.equal(hT, x["h0"])
    got = _backward(x)
    assert torch.equal(got[8], x["dhT"]) and not got[2].any() and not got[5].any() and not got[7].any()


def test_autograd(gpu_lib):
    x = gpu(scan_inputs(14, 2, 90, 72, 16, "bf16", 2))
    names = (*IN, *HOW)
    leaves = {n: x[n].requires_grad_() for n in names}
    y, hT = N.selective_scan(*(leaves[n] for n in IN), **{n: leaves[n] for n in HOW})
    d = torch.autograd.grad([y, hT], [leaves[n] for n in names], [x["dy"], x["dhT"]])
    with torch.no_grad():
        want = dict(zip(NAMES, _backward(x)))
    for n, g in zip(names, d):
        assert torch.equal(g, want["d" + n]), n
    y, _ = N.selective_scan(*(leaves[n] for n in IN))
    with pytest.raises(RuntimeError):
        torch.autograd.grad(torch.autograd.grad(y.float().sum(), leaves["u"], create_graph=True)[0].float().sum(), leaves["u"])


def test_same_bits_every_time(gpu_lib):
    x = gpu(scan_inputs(15, 2, 700, 136, 16, "bf16", 2))
    first = (*_forward(x), *_backward(x))
    for _ in range(3):
        for a, b in zip(first, (*_forward(x), *_backward(x))):
            assert torch.equal(a, b)


def test_refusals(gpu_lib):
    x = gpu(scan_inputs(16, 1, 8, 64, 16, "bf16", 1))
    args = [x[n] for n in IN]
    with pytest.raises(ValueError, match="dt has dtype"):
        N.selective_scan_fwd(args[0], args[1].float(), *args[2:])
    with pytest.raises(ValueError, match="A has dtype"):
        N.selective_scan_fwd(*args[:2], args[2].bfloat16(), *args[3:])
    with pytest.raises(ValueError, match="B has shape"):
        N.selective_scan_fwd(*args[:3], args[3][..., :8].contiguous(), args[4])
    with pytest.raises(ValueError, match="the state has shape"):
        N.selective_scan_fwd(*args, h0=torch.zeros((2, 64, 16), device=DEV))
    with pytest.raises(ValueError, match="batch must be 1"):
        N.selective_scan_fwd(*(t.expand(2, -1, -1) if t.dim() == 3 else t for t in args), cu_seqlens=cu_of([0, 8]))
    with pytest.raises(N.DeltaNetError, match="WORKSPACE"):
        N.selective_scan_bwd(*args, x["dy"], workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
    with pytest.raises(N.DeltaNetError, match="ALIASING"):
        N.selective_scan_fwd(*args, y=x["u"])
