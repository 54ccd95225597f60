"""The selective scan's kernel forms that a batch's or a packed row's sizes choose: packed
sequences in calls that are not cut, with and without the gate, of every number of states.
Bounds: those of the scan's own tests.  (The wide rows' dB and dC are sums over 133 blocks of 64 channels:
6 roundings in a block and 132 of blocks, beside 2 (31 + 12) of the steps, within the 256.)"""

import pytest

from ssm_cases import PACKED, gpu, scan_inputs
from test_gpu_selective_scan import _check

pytestmark = pytest.mark.gpu
#: (rows, channels, cuts): rows that neither direction cuts (32 at most, or no more than a quarter of the
#: workgroups), that the gradient alone cuts (33 to 80), that both do.
ROWS = {"short": (32, 72, [0, 3, 3, 20, 20, 27]), "one tile": (16, 136, [1, 2, 2, 9, 16]), "full": (31, 8, [0, 16, 31]),
        "wide": (33, 8456, [2, 2, 4, 23, 32]), "gradient cut": (70, 72, [4, 4, 5, 36, 70, 70]), "cut": (150, 72, [0, 0, 33, 34, 131, 140])}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S", [8, 16, 32])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("where", ROWS)
def test_packed(gpu_lib, dtype, S, gate, where):
    L, D, cuts = ROWS[where]
    x = scan_inputs(L + S, 1, L, D, S, dtype, len(cuts) - 1, gate=gate)
    _check(x, gpu(x), cuts)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("where", PACKED)
def test_packed_32_states(gpu_lib, dtype, where):
    L, cuts = PACKED[where]
    x = scan_inputs(L, 1, L, 72, 32, dtype, len(cuts) - 1)
    _check(x, gpu(x), cuts)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("S", [8, 16, 32])
@pytest.mark.parametrize("B,L,D", [(2, 1, 24), (3, 20, 72), (2, 47, 64), (1, 150, 136)])
def test_batch_without_a_gate(gpu_lib, dtype, S, B, L, D):
    x = scan_inputs(L + S, B, L, D, S, dtype, B, gate=False)
    _check(x, gpu(x))


@pytest.mark.parametrize("S,gate", [(16, False), (16, True), (32, False), (32, True)])
@pytest.mark.parametrize("B,L,D", [(2, 33, 264), (1, 400, 1024), (9, 130, 1024), (33, 40, 1024), (257, 40, 72)])
def test_rules_of_the_cut_with_more_states(gpu_lib, S, gate, B, L, D):
    x = scan_inputs(L, B, L, D, S, "bf16", B, gate=gate)
    _check(x, gpu(x))
