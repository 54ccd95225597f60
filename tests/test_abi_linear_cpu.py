"""Refusals of the gated linear recurrence and of the q / k norm with rotation:
every check answers before any HIP call (the addresses below are never
dereferenced; nothing is launched)."""

import ctypes

import pytest

from deltanet_delta_rule_chunk_amd import binding

OK, NULL, SHAPE, UNSUP, ALIGN, ALIAS, WS, HIP = range(8)
F32, BF16 = 0, 1
BASE, MB = 1 << 40, 1 << 20
AT = lambda n: BASE + n * 100 * MB  # noqa: E731


@pytest.fixture(scope="module")
def lib():
    return binding.load()


def _fwd(lib, q=AT(0), k=AT(1), v=AT(2), g=AT(3), S0=None, o=AT(4), Sf=AT(5), B=1, H=4, Hqk=2,
         L=256, dk=64, dv=64, it=BF16, ot=F32, ws=AT(6), wb=1 << 40):
    return lib.deltanet_linear_chunk_fwd(q, k, v, g, S0, o, Sf, B, H, Hqk, L, dk, dv, it, ot, ws,
                                         wb, None)


def test_linear_fwd_refusals(lib):
    for name in ("q", "k", "v", "o"):
        assert _fwd(lib, **{name: None}) == NULL
    assert _fwd(lib, B=0) == SHAPE
    assert _fwd(lib, Hqk=3) == SHAPE       # 4 heads do not share 3
    assert _fwd(lib, Hqk=8) == SHAPE
    assert _fwd(lib, Hqk=0) == SHAPE
    assert _fwd(lib, L=-1) == SHAPE
    assert _fwd(lib, dk=96) == UNSUP
    assert _fwd(lib, dv=256) == UNSUP
    assert _fwd(lib, it=2) == UNSUP
    assert _fwd(lib, ot=7) == UNSUP
    assert _fwd(lib, B=20000, H=4, Hqk=4) == UNSUP
    assert _fwd(lib, L=2 ** 31 - 1) == UNSUP
    for name, at in (("q", 0), ("g", 3), ("o", 4), ("Sf", 5), ("ws", 6)):
        assert _fwd(lib, **{name: AT(at) + 8}) == ALIGN
    assert _fwd(lib, o=AT(2)) == ALIAS
    assert _fwd(lib, Sf=AT(3)) == ALIAS
    assert _fwd(lib, Sf=AT(4)) == ALIAS
    assert _fwd(lib, S0=AT(7), Sf=AT(7) + 16) == ALIAS
    assert _fwd(lib, L=4096, ws=AT(1)) == ALIAS
    need = lib.deltanet_linear_chunk_fwd_workspace_bytes(1, 4, 2, 4096, 64, 64, BF16)
    assert need > 0
    assert _fwd(lib, L=4096, wb=need - 1) == WS
    assert lib.deltanet_linear_chunk_fwd_workspace_bytes(1, 4, 3, 4096, 64, 64, BF16) == 0
    assert lib.deltanet_linear_chunk_fwd_workspace_bytes(1, 4, 2, 0, 64, 64, BF16) == 0
    assert lib.deltanet_last_hip_error() == 0


def _bwd(lib, q=AT(0), k=AT(1), v=AT(2), g=AT(3), S0=None, dO=AT(4), dSf=None, dq=AT(5), dk_=AT(6),
         dv_=AT(7), dg=AT(8), dS0=AT(9), B=1, H=4, Hqk=2, L=256, dk=64, dv=64, it=BF16, ws=AT(10),
         wb=1 << 40):
    return lib.deltanet_linear_chunk_bwd(q, k, v, g, S0, dO, dSf, dq, dk_, dv_, dg, dS0, B, H, Hqk,
                                         L, dk, dv, it, ws, wb, None)


def test_linear_bwd_refusals(lib):
    for name in ("q", "k", "v", "dO", "dq", "dk_", "dv_"):
        assert _bwd(lib, **{name: None}) == NULL
    assert _bwd(lib, g=None) == NULL                 # a gradient of a decay that is not there
    assert _bwd(lib, Hqk=3) == SHAPE
    assert _bwd(lib, dk=32) == UNSUP
    assert _bwd(lib, dq=AT(5) + 4) == ALIGN
    assert _bwd(lib, dq=AT(0)) == ALIAS
    assert _bwd(lib, dS0=AT(8)) == ALIAS
    assert _bwd(lib, ws=AT(4)) == ALIAS
    need = lib.deltanet_linear_chunk_bwd_workspace_bytes(1, 4, 2, 256, 64, 64, BF16)
    assert need > 0 and _bwd(lib, wb=need - 1) == WS
    assert lib.deltanet_linear_chunk_bwd_workspace_bytes(1, 4, 2, 256, 64, 65, BF16) == 0
    assert lib.deltanet_last_hip_error() == 0


def _dec(lib, q=AT(0), k=AT(1), v=AT(2), g=AT(3), S=AT(4), o=AT(5), B=2, H=6, Hqk=3, dk=128, dv=64,
         it=BF16, ot=F32):
    return lib.deltanet_linear_decode_step(q, k, v, g, S, o, B, H, Hqk, dk, dv, it, ot, None)


def test_linear_decode_refusals(lib):
    for name in ("q", "k", "v", "S", "o"):
        assert _dec(lib, **{name: None}) == NULL
    assert _dec(lib, Hqk=4) == SHAPE
    assert _dec(lib, B=0) == SHAPE
    assert _dec(lib, B=1 << 28, H=1, Hqk=1) == UNSUP
    assert _dec(lib, dk=100) == UNSUP
    assert _dec(lib, S=AT(4) + 4) == ALIGN
    assert _dec(lib, S=AT(3)) == ALIAS
    assert _dec(lib, o=AT(4)) == ALIAS
    assert lib.deltanet_last_hip_error() == 0


def _ints(*x):
    return (ctypes.c_int * len(x))(*x)


def _str(*x):
    return (ctypes.c_longlong * 3)(*x)


def _qk(lib, q=AT(0), qs=None, k=AT(1), ks=None, qw=AT(2), kw=AT(3), pos=AT(4), inv=AT(5), sec=None,
        axes=1, qh=AT(6), kh=AT(7), B=2, Hq=4, Hk=2, L=10, d=128, drot=128, norm=1, inter=0,
        eps=1e-6, dt=BF16):
    return lib.deltanet_qk_norm_rope(q, qs, k, ks, qw, kw, pos, inv, sec, axes, qh, kh, B, Hq, Hk,
                                     L, d, drot, norm, inter, eps, dt, None)


def _qk_bwd(lib, q=AT(0), qs=None, k=AT(1), ks=None, qw=AT(2), kw=AT(3), pos=AT(4), inv=AT(5),
            sec=None, axes=1, dqh=AT(6), dkh=AT(7), dq=AT(8), dqs=None, dk=AT(9), dks=None,
            dqw=AT(10), dkw=AT(11), B=2, Hq=4, Hk=2, L=10, d=128, drot=128, norm=1, inter=0,
            eps=1e-6, dt=BF16, ws=AT(12), wb=1 << 40):
    return lib.deltanet_qk_norm_rope_bwd(q, qs, k, ks, qw, kw, pos, inv, sec, axes, dqh, dkh, dq,
                                         dqs, dk, dks, dqw, dkw, B, Hq, Hk, L, d, drot, norm, inter,
                                         eps, dt, ws, wb, None)


@pytest.mark.parametrize("call", [_qk, _qk_bwd])
def test_qk_norm_rope_refusals(lib, call):
    for name in ("q", "k", "pos", "inv"):
        assert call(lib, **{name: None}) == NULL
    assert call(lib, B=0) == SHAPE
    assert call(lib, Hq=0) == SHAPE
    assert call(lib, Hk=-1) == SHAPE
    assert call(lib, L=-1) == SHAPE
    assert call(lib, d=96) == UNSUP
    assert call(lib, drot=20) == UNSUP
    assert call(lib, drot=136) == UNSUP
    assert call(lib, drot=-8) == SHAPE
    assert call(lib, dt=3) == UNSUP
    assert call(lib, eps=-1.0) == UNSUP
    assert call(lib, eps=float("nan")) == UNSUP
    assert call(lib, axes=0) == SHAPE
    assert call(lib, axes=3) == NULL                           # sections are required
    assert call(lib, axes=5, sec=_ints(64, 0, 0, 0, 0)) == UNSUP
    assert call(lib, axes=3, sec=_ints(20, 20, 20)) == SHAPE   # 60 of 64 pairs
    assert call(lib, axes=2, sec=_ints(65, -1)) == SHAPE
    assert call(lib, axes=2, sec=_ints(2 ** 31 - 1, 2 ** 31 - 1)) == SHAPE
    assert call(lib, q=AT(0) + 8) == ALIGN
    assert call(lib, qs=_str(5120, 128, 516)) == ALIGN         # rows at 8 bytes
    assert call(lib, ks=_str(5120, -128, 512)) == SHAPE
    assert call(lib, qs=_str(1 << 61, 128, 512)) == UNSUP
    assert lib.deltanet_last_hip_error() == 0


def test_qk_norm_rope_overlaps(lib):
    assert _qk(lib, qh=AT(1)) == ALIAS
    assert _qk(lib, qh=None) == NULL
    assert _qk(lib, kh=AT(6)) == ALIAS
    assert _qk(lib, kh=AT(4)) == ALIAS
    # q_hat inside the extent of q's strided rows
    assert _qk(lib, qs=_str(10 ** 6, 128, 10 ** 5), qh=AT(0) + 2 * 10 ** 6) == ALIAS
    # written rows that share elements
    assert _qk_bwd(lib, dqs=_str(5120, 128, 0)) == ALIAS
    assert _qk_bwd(lib, dqs=_str(5120, 64, 512)) == ALIAS
    assert _qk_bwd(lib, dqs=_str(5120, 128, 384)) == ALIAS
    # the q and k parts of one buffer whose token rows are too short for both
    row = 640
    assert _qk_bwd(lib, dq=AT(8), dqs=_str(10 * row, 128, row), dk=AT(8) + 512 * 2,
                   dks=_str(10 * row, 128, row)) == ALIAS
    # ... that overlap within the row
    row = 768
    assert _qk_bwd(lib, dq=AT(8), dqs=_str(10 * row, 128, row), dk=AT(8) + 384 * 2,
                   dks=_str(10 * row, 128, row)) == ALIAS
    # ... whose k part would run into the next batch's q part
    assert _qk_bwd(lib, dq=AT(8), dqs=_str(9 * row + 512, 128, row), dk=AT(8) + 512 * 2,
                   dks=_str(9 * row + 512, 128, row)) == ALIAS
    # the workspace or a weight's gradient inside that buffer
    assert _qk_bwd(lib, dq=AT(8), dqs=_str(10 * row, 128, row), dk=AT(8) + 512 * 2,
                   dks=_str(10 * row, 128, row), ws=AT(8) + 16) == ALIAS
    assert _qk_bwd(lib, dqw=AT(2)) == ALIAS
    need = lib.deltanet_qk_norm_rope_bwd_workspace_bytes(2, 4, 2, 10, 128, BF16)
    assert need > 0 and _qk_bwd(lib, wb=need - 1) == WS
    assert lib.deltanet_qk_norm_rope_bwd_workspace_bytes(2, 4, 2, 10, 96, BF16) == 0
    assert lib.deltanet_last_hip_error() == 0


def test_calls_without_tokens_launch_nothing(lib):
    assert _fwd(lib, L=0, Sf=None) == OK
    assert _bwd(lib, L=0, dS0=None, q=None, dq=None) == OK
    assert _qk(lib, L=0, q=None, qh=None) == OK
    assert lib.deltanet_last_hip_error() == 0


def test_binding_refuses_wrong_tensors():
    import torch
    x, g = torch.zeros(1, 2, 4, 64), torch.zeros(1, 2, 4)
    with pytest.raises(ValueError, match="GPU"):
        binding.linear_chunk_fwd(x, x, x, g)
    with pytest.raises(ValueError, match="dimensions"):
        binding.linear_chunk_fwd(x[0], x[0], x[0], g[0])
    with pytest.raises(ValueError, match="dimensions"):
        binding.linear_decode_step(x, x, x, g, x)
    with pytest.raises(ValueError, match="GPU"):
        binding.qk_norm_rope(x, x, None, None)
    with pytest.raises(ValueError, match=r"\[B, H, L, d\]"):
        binding.qk_norm_rope(x[0], x[0], None, None)


def test_sizes_beyond_one_launch_are_refused(lib):
    """A launch holds fewer than 2^32 work-items: sizes up to that pass the checks
    of size (and are refused for the overlap here), the next one does not."""
    most = 2 ** 24 - 1                             # workgroups of 256
    assert _dec(lib, B=most, H=1, Hqk=1, S=AT(3)) == ALIAS
    assert _dec(lib, B=most + 1, H=1, Hqk=1, S=AT(3)) == UNSUP
    for call, same in ((_qk, dict(qh=AT(0))), (_qk_bwd, dict(dq=AT(0)))):
        # 32 tokens of 64 elements per workgroup, 16 of 128; up to 4 heads
        for d, rows in ((64, 32), (128, 16)):
            one = dict(B=1, Hq=1, Hk=0, d=d, drot=d, **same)
            assert call(lib, L=most * rows, **one) == ALIAS
            assert call(lib, L=most * rows + 1, **one) == UNSUP
            assert call(lib, L=most // 2 * rows, **dict(one, Hq=5)) == ALIAS
            assert call(lib, L=most // 2 * rows + 1, **dict(one, Hq=5)) == UNSUP
    assert lib.deltanet_last_hip_error() == 0
