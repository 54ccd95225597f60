"""The gradient of the log decays of the gated linear recurrence, token by token.

At token t it is the sum over the pairs (write in front of t, read at t or
behind it) of their terms, all of them under the decay of t.  With A_t the same
sum over the terms' sizes, each term is off by at most E = (L + 512) 2^-24 of
its size (the bound of test_gpu_linear, at t's own A_t and not at the head's
largest)."""

import numpy as np
import pytest
import torch

from deltanet_delta_rule_chunk_amd import binding as N
from oracle import linear_backward
from parity import to64
from test_gpu_linear import _close, _gpu, _inputs, _np

pytestmark = pytest.mark.gpu


def _gradient(x):
    g = _gpu(x)
    got = N.linear_chunk_bwd(g["q"], g["k"], g["v"], g["g"], g["S0"], g["dO"], g["dS"])[3]
    names = ("q", "k", "v", "g", "S0", "dO", "dS")
    want = linear_backward(*(_np(x)[n] for n in names))[3]
    size = linear_backward(*(_np(x, True)[n] for n in names))[3]
    return got, want, size


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("at", [1, 15, 16, 30, 47, 50, 63])
def test_one_strong_token_among_usual_ones(gpu_lib, at, dt, dk, dv):
    """Its gradient is a millionth of its neighbours': pairs on one side of it
    may not enter and leave again."""
    x = _inputs(70 + at, 2, 2, 1, 64, dk, dv, dt, False, "usual")
    x["g"][..., at] = -14.0
    got, want, size = _gradient(x)
    assert (size[..., at] < 1e-4 * size.max(-1)).all()
    _close(got, want, size, torch.float32, 64, "dlog_decay")


@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 128)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("L", [64, 100, 640, 1500])
def test_strong_decays_with_states_at_both_ends(gpu_lib, L, dt, dk, dv):
    """At decays of e^-8 and below a chunk lets nothing through: what the last
    state and its gradient have in common may not reach its tokens."""
    got, want, size = _gradient(_inputs(80, 1, 2, 2, L, dk, dv, dt, True, "strong"))
    _close(got, want, size, torch.float32, L, "dlog_decay")


def _packed(seed, L, starts, dt, states=True):
    x = _gpu(_inputs(seed, 1, 2, 1, L, 64, 64, dt, states, "usual"))
    for t in starts:
        x["g"][..., t] = -float("inf")
    return x


def _decay_gradient(x):
    return N.linear_chunk_bwd(x["q"], x["k"], x["v"], x["g"], x["S0"], x["dO"], x["dS"])[3]


PACKED = [
    # length, starts of the documents behind the first; the third (or the second) one changes
    (64, (20, 41)),
    (128, (64, 100)),
    (500, (200, 301)),
    (700, (64, 128, 129, 640)),
    (3000, (1, 700, 1987, 2999)),
    (20000, (3, 9000, 9010, 15000)),
]


@pytest.mark.parametrize("L,starts", PACKED, ids=[str(p[0]) for p in PACKED])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("times", [0.0, 30.0, 300.0])
def test_a_documents_decay_gradient_is_its_own(gpu_lib, times, dt, L, starts):
    """Documents packed in a row: whatever one of them holds, the decay's gradient
    of the others stays the same bit for bit, and it is 0 in one without loss."""
    x = _packed(81, L, starts, dt)
    want = _decay_gradient(x)
    ends = (0, *starts, L)
    i = 2 if len(starts) > 2 else 1
    at = slice(ends[i], ends[i + 1])
    for n in ("dO",) if times == 0.0 else ("q", "k", "v", "dO"):
        x[n][:, :, at] *= times
    got = _decay_gradient(x)
    for lo, hi in zip(ends, ends[1:]):
        if lo != at.start:
            assert torch.equal(got[..., lo:hi], want[..., lo:hi]), (lo, hi)
    if times == 0.0:
        assert not got[..., at].any()
    # The states at both ends belong to the first and the last document.
    x["S0"] *= 50
    x["dS"] *= 50
    far = _decay_gradient(x)
    inner = slice(starts[0], starts[-1])
    assert torch.equal(far[..., inner], got[..., inner])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_documents_of_unlike_sizes_keep_their_accuracy(gpu_lib, dt):
    """One document 300 times as large as its neighbours, which are as exact as alone."""
    L, starts = 300, (90, 130, 200)
    x = _inputs(82, 1, 2, 1, L, 64, 64, dt, True, "usual")
    for t in starts:
        x["g"][..., t] = -float("inf")
    for n in ("q", "k", "v", "dO"):
        x[n][:, :, 90:130] *= 300
    got, want, size = _gradient(x)
    for lo, hi in zip((0, *starts), (*starts, L)):
        most = size[..., lo:hi].max(-1, keepdims=True) * np.ones_like(size[..., lo:hi])
        _close(got[..., lo:hi], want[..., lo:hi], most, torch.float32, L, "dlog_decay", 2 * L / 64 + 3)
