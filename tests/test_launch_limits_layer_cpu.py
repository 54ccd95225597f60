"""Sizes at the ends of what one launch takes, 2^32 - 1 work-items: refused beyond them, taken up to
them (answered before any HIP call)."""

from deltanet_delta_rule_chunk_amd import binding as N
from test_abi_layer_cpu import ALIAS, UNSUP, _norm, _norm_bwd, _scan_bwd, lib  # noqa: F401


def test_scan_gradient_sums_of_many_channels(lib):
    """16 columns of dA, dD and the bias's gradient per workgroup of 256."""
    bytes_of = lib.deltanet_selective_scan_bwd_workspace_bytes
    for S in (8, 16, 32):
        most = min((2 ** 32 - 1) // 256 * 16 // (S + 2) // 8 * 8, 2 ** 24)
        assert bytes_of(1, 1, most, S, 0, 1) > 0
        # (Accepted sizes get as far as the overlap of the addresses that stand for tensors.)
        assert _scan_bwd(lib, B=1, L=1, D=most, N=S) == ALIAS
        assert bytes_of(1, 1, most + 8, S, 0, 1) == 0
        assert _scan_bwd(lib, B=1, L=1, D=most + 8, N=S) == UNSUP


def test_norm_rows_are_counted_by_workgroups(lib):
    """Rows of up to 128 elements go 16 to a workgroup of 256, of up to 2048 elements 4."""
    blocks = (2 ** 32 - 1) // 256
    for D, rows_each in ((64, 16), (128, 16), (136, 4), (2048, 4), (2056, 1), (8192, 1)):
        most = blocks * rows_each
        assert lib.deltanet_add_rms_norm_bwd_workspace_bytes(most, D) > 0
        assert _norm(lib, rows=most, D=D) == ALIAS and _norm_bwd(lib, rows=most, D=D) == ALIAS
        assert lib.deltanet_add_rms_norm_bwd_workspace_bytes(most + 1, D) == 0
        assert _norm(lib, rows=most + 1, D=D) == UNSUP and _norm_bwd(lib, rows=most + 1, D=D) == UNSUP
    assert lib.deltanet_add_rms_norm_bwd_workspace_bytes(2 ** 31 - 1, 32768) == 0
