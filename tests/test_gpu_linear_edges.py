"""The gated linear recurrence where memory and rows end: what lies behind a
tensor's last row, documents that a wipe separates, states that are not finite."""

import pytest
import torch

from deltanet_delta_rule_chunk_amd import binding as N
from test_gpu_linear import _gpu, _inputs

pytestmark = pytest.mark.gpu
NAMES = ("q", "k", "v", "g", "S0", "dO", "dS")


def _followed_by_nan(t):
    """The same tensor at the start of an allocation that goes on with a chunk's
    rows and more of NaN."""
    buf = torch.full((t.numel() + 128 * 128,), float("nan"), dtype=t.dtype, device=t.device)
    buf[:t.numel()] = t.flatten()
    return buf[:t.numel()].view(t.shape)


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("L", [1, 17, 66, 200])
def test_rows_behind_a_ragged_head_do_not_show(gpu_lib, L, dt, dk, dv):
    """A ragged last chunk reads nothing behind its head: with NaN there every
    output and gradient is what it is without."""
    x = _gpu(_inputs(60, 1, 2, 1, L, dk, dv, dt, True, "usual"))
    y = {n: _followed_by_nan(t) for n, t in x.items()}

    def call(x):
        return (*N.linear_chunk_fwd(*(x[n] for n in NAMES[:5])),
                *N.linear_chunk_bwd(*(x[n] for n in NAMES)))

    for i, (a, b) in enumerate(zip(call(x), call(y))):
        assert torch.isfinite(b).all() and torch.equal(a, b), i


# (heads, length): sequences that are cut into segments of one chunk, of several, not at all
SPLITS = [(1, 200), (2, 700), (16, 2000), (200, 300), (2, 64)]


@pytest.mark.parametrize("H,L", SPLITS)
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("gates", ["wiping", "strong", "usual"])
def test_a_state_that_is_not_finite_stays_so(gpu_lib, gates, dt, H, L):
    """However the sequence is cut, also where a segment starts with a wipe or its
    decays leave nothing of what enters it."""
    x = _gpu(_inputs(61, 1, H, 1, L, 64, 64, dt, True, gates))
    x["g"][..., 0] = -0.1
    if gates == "wiping":
        x["g"][..., 64::64] = -float("inf")
    x["v"][:, :, 10] = float("nan")
    o, S = N.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["S0"])
    assert not torch.isfinite(o[:, :, 10:]).any() and not torch.isfinite(S).any()
    # ... nor does the gradient of the states in front of a row whose gradient is not.
    x["v"][:, :, 10] = 1
    x["dO"][:, :, L - 1] = float("nan")
    dS0 = N.linear_chunk_bwd(*(x[n] for n in NAMES))[4]
    assert not torch.isfinite(dS0).any()
