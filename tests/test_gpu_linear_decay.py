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
