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
