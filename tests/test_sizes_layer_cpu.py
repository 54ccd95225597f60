"""Sizes past a C int in the state space layer's calls: refused as they are, not cut to
their low 32 bits (tensors without memory stand for those that a card holds)."""

import pytest
import torch

from deltanet_delta_rule_chunk_amd import binding as N

MANY = 2 ** 32 + 5  # 5, once cut


def _meta(*shape, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="meta")


def _f32(*shape):
    return _meta(*shape, dtype=torch.float32)


def _conv(B, L, D):
    x, w, kept = _meta(B, L, D), _f32(D, 4), _meta(B, 3, D)
    return [lambda: N.short_conv_fwd(x, w), lambda: N.short_conv_bwd(x, w, None, None, x),
            lambda: N.short_conv(x, w), *([lambda: N.short_conv_step(x[:, 0], w, None, kept)] if L == 1 else [])]


def _scan(B, L, D):
    u, A, few, h = _meta(B, L, D), _f32(D, 8), _meta(B, L, 8), _f32(B, D, 8)
    return [lambda: N.selective_scan_fwd(u, u, A, few, few), lambda: N.selective_scan_bwd(u, u, A, few, few, u),
            lambda: N.selective_scan(u, u, A, few, few),
            *([lambda: N.selective_scan_step(u[:, 0], u[:, 0], A, few[:, 0], few[:, 0], h)] if L == 1 else [])]


def _norm(*shape):
    x = _meta(*shape)
    return [lambda: N.add_rms_norm(x, x, None), lambda: N.add_rms_norm_fp8(x, None, None),
            lambda: N.add_rms_norm_bwd(x, None, x), lambda: N.residual_norm(x, x, None)]


@pytest.mark.parametrize("op,shape", [
    (_conv, (MANY, 1, 8)), (_conv, (1, MANY, 8)), (_conv, (1, 1, 2 ** 32 + 8)), (_conv, (2 ** 31, 1, 8)),
    (_scan, (MANY, 1, 8)), (_scan, (1, MANY, 8)), (_scan, (1, 1, 2 ** 32 + 8)), (_scan, (1, 2 ** 31, 8)),
    (_norm, (MANY, 8)), (_norm, (2 ** 16, 2 ** 16 + 1, 8)), (_norm, (1, 2 ** 32 + 8)), (_norm, (2 ** 31, 8))])
def test_sizes_past_a_c_int(op, shape):
    for call in op(*shape):
        with pytest.raises(N.DeltaNetError, match=r"UNSUPPORTED.*2\^31 - 1"):
            call()


@pytest.mark.parametrize("op,shape", [(_conv, (2 ** 31 - 1, 1, 8)), (_scan, (1, 2 ** 31 - 1, 8)), (_norm, (2 ** 31 - 1, 8))])
def test_the_largest_c_int_is_for_the_library_to_judge(op, shape):
    for call in op(*shape):
        with pytest.raises(ValueError, match="GPU"):
            call()
