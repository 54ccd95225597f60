"""The short causal convolution against the fp64 one, forward, backward and token by token.

Bounds, in fp32 roundings of the terms' magnitudes.  Forward: K + 1 additions and
products of the tap sum; the sigmoid's exponent is off by 1.5 |p| 2^-24 of it (times
p^2 s (1 - s) <= |p|), its three operations by 5: 20 covers K = 4.  Gradients of x:
the same through silu' (|silu''| <= 1/2) and K products: 30.  Of the weights: 30 and one
rounding per row of a thread's run, at most 256.
"""

import numpy as np
import pytest
import torch

from deltanet_delta_rule_chunk_amd import binding as N
from oracle import conv_backward, conv_forward, spans_of
from ssm_cases import DEV, PACKED, TYPES, close, conv_inputs, cu_of, f64, gpu

pytestmark = pytest.mark.gpu


def _sizes(x, spans, silu):
    a = {k: None if v is None else np.abs(v) for k, v in x.items()}
    y, s = conv_forward(a["x"], a["weight"], a["bias"], a["state0"], spans, False)
    return 1.1 * y + (1.0 if silu else 0.0) * 1e-3, s


def _check(x, g, cuts, silu):
    B, L, D = x["x"].shape
    e, spans = {k: f64(v) for k, v in x.items()}, spans_of(*x["x"].shape[:2], cuts)
    cu = cu_of(cuts)
    y, state = N.short_conv_fwd(g["x"], g["weight"], g["bias"], g["state0"], silu=silu, cu_seqlens=cu)
    want, kept = conv_forward(e["x"], e["weight"], e["bias"], e["state0"], spans, silu)
    size, _ = _sizes(e, spans, silu)
    close(y, want, size, 20, "y")
    assert np.array_equal(f64(state), kept)
    got = N.short_conv_bwd(g["x"], g["weight"], g["bias"], g["state0"], g["dy"], g["dstate"], silu=silu, cu_seqlens=cu)
    how = (e["weight"], e["bias"], e["state0"], e["dy"], e["dstate"], spans, silu)
    want, size = conv_backward(e["x"], *how), conv_backward(e["x"], *how, size=True)
    units = {"dx": 30, "dweight": 30 + min(L, 256), "dbias": 30 + min(L, 256), "dstate0": 30}
    for i, (name, u) in enumerate(units.items()):
        if got[i] is not None:
            close(got[i], want[i], size[i], u, name)
    assert (got[2] is None) == (g["bias"] is None)
    outside = np.ones((B, L), bool)
    for row, lo, hi in spans:
        outside[row, lo:hi] = False
    assert not y.cpu()[torch.from_numpy(outside)].any() and not got[0].cpu()[torch.from_numpy(outside)].any()


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [2, 3, 4])
@pytest.mark.parametrize("B,L,D", [(1, 1, 8), (3, 2, 24), (2, 3, 64), (2, 16, 136), (2, 17, 520), (1, 300, 40)])
def test_batch(gpu_lib, dtype, K, B, L, D):
    x = conv_inputs(L, B, L, D, K, dtype, B)
    _check(x, gpu(x), None, True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("where", PACKED)
@pytest.mark.parametrize("K", [2, 4])
def test_packed(gpu_lib, dtype, where, K):
    L, cuts = PACKED[where]
    x = conv_inputs(L + K, 1, L, 72, K, dtype, len(cuts) - 1)
    _check(x, gpu(x), cuts, True)


@pytest.mark.parametrize("state,bias,silu", [(False, True, True), (True, False, False), (False, False, False)])
def test_forms(gpu_lib, state, bias, silu):
    for cuts in (None, [0, 2, 2, 45, 60]):
        x = conv_inputs(4, 1, 61, 24, 4, "bf16", 1 if cuts is None else 4, state, bias)
        _check(x, gpu(x), cuts, silu)


def test_long_runs(gpu_lib):
    """Enough rows for the backward's longest runs."""
    x = conv_inputs(6, 2, 1500, 264, 4, "bf16", 2)
    _check(x, gpu(x), None, True)


def test_rows_out_of_a_projection(gpu_lib):
    x = conv_inputs(8, 2, 37, 64, 4, "bf16", 2)
    g = gpu(x)
    rows = torch.randn((2, 37, 3 * 64), device=DEV).to(torch.bfloat16)
    rows[..., 64:128] = g["x"]
    g["x"] = rows[..., 64:128]
    _check(x, g, None, True)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [2, 3, 4])
def test_tokens_one_by_one(gpu_lib, dtype, K):
    x = conv_inputs(9, 5, 7, 40, K, dtype, 5)
    g = gpu(x)
    y, state = N.short_conv_fwd(g["x"], g["weight"], g["bias"], g["state0"])
    kept = g["state0"].clone()
    rows = [N.short_conv_step(g["x"][:, t], g["weight"], g["bias"], kept) for t in range(7)]
    assert torch.equal(torch.stack(rows, 1), y) and torch.equal(kept, state)


def test_pieces_of_a_sequence_are_the_whole(gpu_lib):
    x = gpu(conv_inputs(10, 2, 90, 64, 4, "bf16", 2))
    y, state = N.short_conv_fwd(x["x"], x["weight"], x["bias"], x["state0"])
    s, parts = x["state0"], []
    for lo, hi in ((0, 1), (1, 3), (3, 50), (50, 90)):
        p, s = N.short_conv_fwd(x["x"][:, lo:hi], x["weight"], x["bias"], s)
        parts.append(p)
    assert torch.equal(torch.cat(parts, 1), y) and torch.equal(s, state)


def test_what_is_not_finite_stays_in_its_sequence(gpu_lib):
    """A sequence of NaN, kept rows of NaN in front of it and padding of NaN: the others'
    outputs do not change by a bit, and rows of no sequence are zeros."""
    cuts = [0, 10, 21, 40]
    x = gpu(conv_inputs(11, 1, 48, 64, 4, "bf16", 3))
    cu = cu_of(cuts)
    call = lambda v: (*N.short_conv_fwd(v["x"], v["weight"], v["bias"], v["state0"], cu_seqlens=cu),  # noqa: E731
                      *N.short_conv_bwd(v["x"], v["weight"], v["bias"], v["state0"], v["dy"], v["dstate"], cu_seqlens=cu))
    want = call(x)
    bad = {k: v.clone() for k, v in x.items()}
    for n in ("x", "dy"):
        bad[n][:, 10:21] = float("nan")
        bad[n][:, 40:] = float("inf")
    bad["state0"][1] = float("nan")
    got = call(bad)
    keep = [i for i in range(40) if not 10 <= i < 21]
    for i in (0, 2):
        assert torch.equal(got[i][:, keep], want[i][:, keep]) and not got[i][:, 40:].any()
    for i in (1, 5):
        assert torch.equal(got[i][[0, 2]], want[i][[0, 2]])
    assert got[3].isnan().all()  # the weights' gradient sums over all sequences


def test_cuts_that_fall_or_leave_the_rows_stay_in_bounds(gpu_lib):
    x = gpu(conv_inputs(12, 1, 40, 64, 4, "bf16", 4))
    for cuts in ([0, 30, 10, 50, 40], [-7, 5, 5, 2 ** 31 - 1, 3], [50, 60, 70, 80, 90]):
        y, s = N.short_conv_fwd(x["x"], x["weight"], x["bias"], x["state0"], cu_seqlens=cu_of(cuts))
        d = N.short_conv_bwd(x["x"], x["weight"], x["bias"], x["state0"], x["dy"], x["dstate"], cu_seqlens=cu_of(cuts))
        torch.cuda.synchronize()
        assert all(torch.isfinite(t.float()).all() for t in (y, *d))


def test_no_tokens(gpu_lib):
    x = gpu(conv_inputs(15, 2, 0, 64, 4, "bf16", 2))
    y, state = N.short_conv_fwd(x["x"], x["weight"], x["bias"], x["state0"])
    assert y.shape == (2, 0, 64) and torch.equal(state, x["state0"])
    dx, dw, db, ds = N.short_conv_bwd(x["x"], x["weight"], x["bias"], x["state0"], x["dy"], x["dstate"])
    assert dx.shape == (2, 0, 64) and not dw.any() and not db.any() and torch.equal(ds, x["dstate"])


def test_autograd(gpu_lib):
    x = conv_inputs(13, 2, 19, 24, 4, "f32", 2)
    g = gpu(x)
    leaves = [g[n].requires_grad_() for n in ("x", "weight", "bias", "state0")]
    y, s = N.short_conv(*leaves)
    d = torch.autograd.grad((y * g["dy"]).sum() + (s * g["dstate"]).sum(), leaves)
    want = N.short_conv_bwd(*(g[n].detach() for n in ("x", "weight", "bias", "state0", "dy", "dstate")))
    for a, b in zip(d, want):
        assert torch.equal(a, b)
    y, _ = N.short_conv(leaves[0], leaves[1])
    with pytest.raises(RuntimeError):
        torch.autograd.grad(torch.autograd.grad(y.sum(), leaves[0], create_graph=True)[0].sum(), leaves[0])


def test_refusals(gpu_lib):
    x = gpu(conv_inputs(14, 1, 8, 64, 4, "bf16", 1))
    with pytest.raises(ValueError, match="state0 has shape"):
        N.short_conv_fwd(x["x"], x["weight"], x["bias"], x["state0"][:, :2].contiguous())
    with pytest.raises(ValueError, match="state0 has dtype"):
        N.short_conv_fwd(x["x"], x["weight"], x["bias"], x["state0"].float())
    with pytest.raises(ValueError, match="cu_seqlens has dtype"):
        N.short_conv_fwd(x["x"], x["weight"], cu_seqlens=torch.tensor([0, 8], device=DEV))
    with pytest.raises(ValueError, match="cu_seqlens must be on the GPU"):
        N.short_conv_fwd(x["x"], x["weight"], cu_seqlens=torch.tensor([0, 8], dtype=torch.int32))
    with pytest.raises(TypeError, match="dtype"):
        N.short_conv_fwd(x["x"].half(), x["weight"])
    with pytest.raises(N.DeltaNetError, match="UNSUPPORTED"):
        N.short_conv_fwd(x["x"], torch.zeros((64, 5), device=DEV))
    with pytest.raises(N.DeltaNetError, match="MISALIGNED"):
        N.short_conv_fwd(torch.zeros((1, 8, 68), device=DEV, dtype=torch.bfloat16)[..., 4:], x["weight"])
