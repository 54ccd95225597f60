"""Sizes at the ends of what one launch takes, 2^32 - 1 work-items: refused beyond them, taken up to
them (answered before any HIP call)."""

from deltanet_delta_rule_chunk_amd import binding as N
from test_abi_layer_cpu import ALIAS, UNSUP, _scan_bwd, lib  # noqa: F401


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
