"""How many bits the gated linear recurrence's fp32 results have, in the mean.

Element by element a bound has to allow for every rounding at its worst; in the
mean independent roundings add as the root of their number.  A state is summed
over L / 64 chunks with at most 16 additions each (fp32 inputs: 64 rows, 4 to a
matrix instruction; bf16: 32 rows, 3 pieces), an output over 48 more; with a
rounding of 2^-24 / sqrt(3) in the mean, on partial sums no larger than the
whole, L = 1500 gives sqrt((24 16 + 24 + 48) / 3) 2^-24 = 12.4 2^-24, and the decays' factors
(2^-a, off by a 2^-25 and a step) below 2 2^-24 more.  An operand cut to two bf16
pieces instead leaves 2^-17 of its terms at most, 2.3e-6 = 39 2^-24 in the mean."""

import numpy as np
import pytest
import torch

from deltanet_delta_rule_chunk_amd import binding as N
from oracle import linear_backward, linear_forward
from parity import to64
from test_gpu_linear import _gpu, _inputs, _np

pytestmark = pytest.mark.gpu
BOUND = 16 * 2.0 ** -24

CASES = [
    # B, Hqk, grp, L, dk, dv, dtype, state, gates
    (1, 2, 1, 64, 64, 64, "bf16", False, "usual"),      # what the chunk's own rows give
    (1, 2, 1, 1, 128, 128, "bf16", True, "keep"),       # what the state gives
    (1, 2, 2, 333, 128, 64, "bf16", True, "wiping"),
    (1, 2, 1, 1500, 64, 128, "bf16", True, "usual"),
    (1, 2, 1, 1500, 128, 128, "bf16", False, "none"),   # a state of many segments' sums
    (2, 40, 2, 250, 128, 128, "bf16", True, "usual"),   # one segment
    (1, 2, 1, 1500, 128, 128, "f32", True, "usual"),
    (1, 2, 2, 700, 64, 64, "f32", True, "keep"),
]


def _off(got, want):
    return np.linalg.norm(to64(got) - want) / np.linalg.norm(want)


@pytest.mark.parametrize("case", CASES, ids=["-".join(map(str, c)) for c in CASES])
def test_fp32_results_have_fp32s_bits(gpu_lib, case):
    dt = case[6]
    x = _inputs(90, *case)
    g, e = _gpu(x), _np(x)
    o, S = N.linear_chunk_fwd(g["q"], g["k"], g["v"], g["g"], g["S0"])
    want = linear_forward(e["q"], e["k"], e["v"], e["g"], e["S0"])
    off = {"o": _off(o, want[0]), "S_final": _off(S, want[1])}
    names = ("q", "k", "v", "g", "S0", "dO", "dS")
    got = N.linear_chunk_bwd(*(g[n] for n in names))
    want = linear_backward(*(e[n] for n in names))
    off["dS0"] = _off(got[4], want[4])
    if dt == "f32":
        off.update((n, _off(got[i], want[i])) for i, n in enumerate(("dq", "dk", "dv")))
    print({n: f"{v / 2.0 ** -24:.1f}" for n, v in off.items()})
    assert all(v <= BOUND for v in off.values()), off


def test_a_bf16_output_is_its_fp32_one_rounded(gpu_lib):
    """Two pieces on the way to a bf16 o change its rounding at about
    2^-17 / 2^-8 of the places at most, by one step."""
    x = _gpu(_inputs(91, 2, 4, 1, 700, 128, 128, "bf16", True, "usual"))
    call = lambda t: N.linear_chunk_fwd(x["q"], x["k"], x["v"], x["g"], x["S0"], out_dtype=t)  # noqa: E731
    (o, S), (w, W) = call(torch.bfloat16), call(torch.float32)
    assert torch.equal(S, W)
    other = o != w.bfloat16()
    assert float(other.float().mean()) < 2.0 ** -9
    d = (o.double() - w.double()).abs()
    assert (d <= (2.0 ** -8 + 2.0 ** -16) * w.double().abs() + 2.0 ** -16 * float(w.abs().max())).all()
