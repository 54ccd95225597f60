"""Refusals of the state space layer's operators: every check answers before any HIP
call (the addresses below are never dereferenced; nothing is launched)."""

import ctypes

import pytest
import torch

from deltanet_delta_rule_chunk_amd import binding

OK, NULL, SHAPE, UNSUP, ALIGN, ALIAS, WS, HIP = range(8)
F32, BF16 = 0, 1
BASE, MB = 1 << 40, 1 << 20
AT = lambda n: BASE + n * 100 * MB  # noqa: E731


@pytest.fixture(scope="module")
def lib():
    return binding.load()


def _ll(*x):
    return (ctypes.c_longlong * len(x))(*x)


def _conv(lib, x=AT(0), st=None, w=AT(1), b=AT(2), s0=AT(3), cu=None, y=AT(4), s=AT(5), B=2, L=100,
          D=64, K=4, n=0, silu=1, dt=BF16):
    return lib.deltanet_short_conv_fwd(x, st, w, b, s0, cu, y, s, B, L, D, K, n, silu, dt, None)


def _conv_bwd(lib, x=AT(0), st=None, w=AT(1), b=AT(2), s0=AT(3), cu=None, dy=AT(4), ds=AT(5), dx=AT(6),
              dw=AT(7), db=AT(8), ds0=AT(9), B=2, L=100, D=64, K=4, n=0, silu=1, dt=BF16, ws=AT(10),
              wb=1 << 40):
    return lib.deltanet_short_conv_bwd(x, st, w, b, s0, cu, dy, ds, dx, dw, db, ds0, B, L, D, K, n, silu, dt,
                                       ws, wb, None)


def _conv_step(lib, x=AT(0), st=None, w=AT(1), b=AT(2), s=AT(3), y=AT(4), B=2, D=64, K=4, silu=1, dt=BF16):
    return lib.deltanet_short_conv_step(x, st, w, b, s, y, B, D, K, silu, dt, None)


@pytest.mark.parametrize("call", [_conv, _conv_bwd])
def test_conv_refusals(lib, call):
    for name in ("x", "w"):
        assert call(lib, **{name: None}) == NULL
    assert call(lib, B=0) == SHAPE
    assert call(lib, L=-1) == SHAPE
    assert call(lib, D=0) == SHAPE
    assert call(lib, K=0) == SHAPE
    assert call(lib, D=60) == UNSUP
    for K in (1, 5):
        assert call(lib, K=K) == UNSUP
    assert call(lib, dt=2) == UNSUP
    assert call(lib, L=2 ** 31 - 1) == UNSUP
    assert call(lib, cu=AT(20), n=3) == SHAPE            # packed sequences take one batch row
    assert call(lib, cu=AT(20), B=1, n=0) == SHAPE
    assert call(lib, cu=AT(20) + 2, B=1, n=3) == ALIGN
    assert call(lib, x=AT(0) + 8) == ALIGN
    assert call(lib, w=AT(1) + 4) == ALIGN
    assert call(lib, st=_ll(6400, 68)) == ALIGN          # rows at 8 bytes
    assert call(lib, st=_ll(6400, -64)) == SHAPE
    assert call(lib, st=_ll(1 << 60, 64)) == UNSUP
    assert lib.deltanet_last_hip_error() == 0


def test_conv_overlaps(lib):
    assert _conv(lib, y=None) == NULL
    for at in (0, 1, 2, 3):
        assert _conv(lib, y=AT(at)) == ALIAS
    assert _conv(lib, s=AT(3)) == ALIAS                  # the rows behind are not written over those in front
    assert _conv(lib, s=AT(4)) == ALIAS
    assert _conv(lib, cu=AT(20), B=1, n=3, y=AT(20)) == ALIAS
    assert _conv(lib, st=_ll(10 ** 6, 64 * 64), y=AT(0) + 2 * 10 ** 6) == ALIAS   # inside the strided rows' extent
    for name in ("dy", "dx", "dw"):
        assert _conv_bwd(lib, **{name: None}) == NULL
    assert _conv_bwd(lib, dx=AT(0)) == ALIAS
    assert _conv_bwd(lib, dx=AT(4)) == ALIAS
    assert _conv_bwd(lib, ds0=AT(3)) == ALIAS
    assert _conv_bwd(lib, db=AT(7)) == ALIAS
    assert _conv_bwd(lib, ws=AT(4)) == ALIAS
    need = lib.deltanet_short_conv_bwd_workspace_bytes(2, 100, 64, 4)
    assert need > 0 and _conv_bwd(lib, wb=need - 1) == WS
    for bad in ((2, 100, 60, 4), (2, 100, 64, 5), (0, 100, 64, 4), (2, -1, 64, 4)):
        assert lib.deltanet_short_conv_bwd_workspace_bytes(*bad) == 0
    for name in ("x", "w", "s", "y"):
        assert _conv_step(lib, **{name: None}) == NULL
    assert _conv_step(lib, K=7) == UNSUP
    assert _conv_step(lib, B=0) == SHAPE
    assert _conv_step(lib, st=_ll(68)) == ALIGN
    assert _conv_step(lib, y=AT(3)) == ALIAS
    assert _conv_step(lib, s=AT(0)) == ALIAS
    assert lib.deltanet_last_hip_error() == 0


def _scan(lib, u=AT(0), d=AT(1), Bm=AT(2), Cm=AT(3), z=AT(4), st=None, A=AT(5), sk=AT(6), b=AT(7), h0=AT(8),
          cu=None, y=AT(9), hT=AT(10), B=2, L=100, D=64, N=16, n=0, sp=1, dt=BF16, ws=AT(11), wb=1 << 40):
    return lib.deltanet_selective_scan_fwd(u, d, Bm, Cm, z, st, A, sk, b, h0, cu, y, hT, B, L, D, N, n, sp, dt,
                                           ws, wb, None)


def _scan_bwd(lib, u=AT(0), d=AT(1), Bm=AT(2), Cm=AT(3), z=AT(4), st=None, A=AT(5), sk=AT(6), b=AT(7), h0=AT(8),
              cu=None, dy=AT(9), dhT=AT(10), du=AT(12), dd=AT(13), dB=AT(14), dC=AT(15), dz=AT(16), dA=AT(17),
              dsk=AT(18), db=AT(19), dh0=AT(21), B=2, L=100, D=64, N=16, n=0, sp=1, dt=BF16, ws=AT(11), wb=1 << 40):
    return lib.deltanet_selective_scan_bwd(u, d, Bm, Cm, z, st, A, sk, b, h0, cu, dy, dhT, du, dd, dB, dC, dz, dA,
                                           dsk, db, dh0, B, L, D, N, n, sp, dt, ws, wb, None)


def _scan_step(lib, u=AT(0), d=AT(1), Bm=AT(2), Cm=AT(3), z=AT(4), st=None, A=AT(5), sk=AT(6), b=AT(7), h=AT(8),
               y=AT(9), B=2, D=64, N=16, sp=1, dt=BF16):
    return lib.deltanet_selective_scan_step(u, d, Bm, Cm, z, st, A, sk, b, h, y, B, D, N, sp, dt, None)


@pytest.mark.parametrize("call", [_scan, _scan_bwd, _scan_step])
def test_scan_refusals(lib, call):
    for name in ("u", "d", "Bm", "Cm", "A"):
        assert call(lib, **{name: None}) == NULL
    assert call(lib, B=0) == SHAPE
    assert call(lib, D=-8) == SHAPE
    assert call(lib, N=0) == SHAPE
    assert call(lib, D=68) == UNSUP
    for N in (4, 12, 64):
        assert call(lib, N=N) == UNSUP
    assert call(lib, dt=5) == UNSUP
    for name, at in (("u", 0), ("Bm", 2), ("z", 4), ("A", 5), ("b", 7)):
        assert call(lib, **{name: AT(at) + 8}) == ALIGN
    assert lib.deltanet_last_hip_error() == 0


@pytest.mark.parametrize("call", [_scan, _scan_bwd])
def test_scan_sequence_refusals(lib, call):
    assert call(lib, L=-1) == SHAPE
    assert call(lib, L=2 ** 31 - 1) == UNSUP
    assert call(lib, cu=AT(20), n=3) == SHAPE
    assert call(lib, cu=AT(20), B=1, n=-1) == SHAPE
    assert call(lib, cu=AT(20) + 1, B=1, n=3) == ALIGN
    rows = [6400, 64, 6400, 64, 1600, 16, 1600, 16, 6400, 64]
    for at, bad, want in ((1, 68, ALIGN), (3, -64, SHAPE), (5, 4, ALIGN), (8, 1 << 60, UNSUP)):
        assert call(lib, st=_ll(*(bad if i == at else v for i, v in enumerate(rows)))) == want
    assert lib.deltanet_last_hip_error() == 0


def test_scan_overlaps(lib):
    assert _scan(lib, y=None) == NULL
    for at in (0, 1, 2, 3, 4, 5, 8):
        assert _scan(lib, y=AT(at)) == ALIAS
    assert _scan(lib, hT=AT(8) + 16) == ALIAS            # (h0 itself is allowed, a part of it not)
    assert _scan(lib, hT=AT(5)) == ALIAS
    assert _scan(lib, L=4096, ws=AT(1)) == ALIAS
    need = lib.deltanet_selective_scan_fwd_workspace_bytes(2, 4096, 64, 16, 0, 0)
    assert need > 0 and _scan(lib, L=4096, wb=need - 1) == WS
    packed = lib.deltanet_selective_scan_fwd_workspace_bytes(1, 4096, 64, 16, 1, 9)
    assert packed > 0 and _scan(lib, B=1, L=4096, cu=AT(20), n=9, wb=packed - 1) == WS
    for name in ("dy", "du", "dd", "dB", "dC", "dz", "dA"):
        assert _scan_bwd(lib, **{name: None}) == NULL
    for name, at in (("du", 0), ("dd", 12), ("dB", 2), ("dz", 9), ("dA", 5), ("dh0", 8), ("dh0", 10), ("db", 18)):
        assert _scan_bwd(lib, **{name: AT(at)}) == ALIAS
    assert _scan_bwd(lib, ws=AT(9)) == ALIAS
    need = lib.deltanet_selective_scan_bwd_workspace_bytes(2, 100, 64, 16, 0, 0)
    assert need > 0 and _scan_bwd(lib, wb=need - 1) == WS
    for fn in (lib.deltanet_selective_scan_fwd_workspace_bytes, lib.deltanet_selective_scan_bwd_workspace_bytes):
        for bad in ((2, 100, 60, 16, 0, 0), (2, 100, 64, 20, 0, 0), (0, 100, 64, 16, 0, 0), (2, 100, 64, 16, 1, 4),
                    (1, 100, 64, 16, 1, 0)):
            assert fn(*bad) == 0
    assert _scan_step(lib, h=None) == NULL
    assert _scan_step(lib, y=None) == NULL
    assert _scan_step(lib, y=AT(8)) == ALIAS
    assert _scan_step(lib, h=AT(5)) == ALIAS
    assert _scan_step(lib, st=_ll(68, 64, 16, 16, 64)) == ALIGN
    assert lib.deltanet_last_hip_error() == 0


def _norm(lib, x=AT(0), r=AT(1), w=AT(2), t=AT(3), y=AT(4), s=None, rows=10, D=64, eps=1e-6, dt=BF16, rt=BF16):
    return lib.deltanet_add_rms_norm(x, r, w, t, y, s, rows, D, eps, dt, rt, None)


def _norm_bwd(lib, t=AT(0), w=AT(1), dy=AT(2), dt_=AT(3), dx=AT(4), dr=None, dw=AT(5), rows=10, D=64, eps=1e-6,
              dt=BF16, rt=BF16, ws=AT(6), wb=1 << 40):
    return lib.deltanet_add_rms_norm_bwd(t, w, dy, dt_, dx, dr, dw, rows, D, eps, dt, rt, ws, wb, None)


def test_norm_refusals(lib):
    for call in (_norm, _norm_bwd):
        assert call(lib, rows=-1) == SHAPE
        assert call(lib, D=0) == SHAPE
        assert call(lib, D=68) == UNSUP
        assert call(lib, D=32776) == UNSUP
        assert call(lib, dt=3) == UNSUP
        assert call(lib, dt=F32, rt=BF16) == UNSUP
        assert call(lib, eps=-1.0) == UNSUP
        assert call(lib, eps=float("nan")) == UNSUP
        assert call(lib, w=AT(2) + 4) == ALIGN
    assert _norm(lib, x=None) == NULL
    assert _norm(lib, y=None) == NULL
    assert _norm(lib, t=None) == NULL                    # a residual without its sum
    assert _norm(lib, r=None) == NULL
    assert _norm(lib, y=AT(0)) == ALIAS
    assert _norm(lib, y=AT(3)) == ALIAS
    assert _norm(lib, t=AT(1) + 16) == ALIAS
    assert _norm(lib, t=AT(0), rt=F32) == ALIAS          # x and the sum differ in type
    assert _norm(lib, s=AT(4)) == ALIAS
    for name in ("t", "dy", "dx"):
        assert _norm_bwd(lib, **{name: None}) == NULL
    assert _norm_bwd(lib, dx=AT(2)) == ALIAS
    assert _norm_bwd(lib, dr=AT(4)) == ALIAS
    assert _norm_bwd(lib, ws=AT(3)) == ALIAS
    need = lib.deltanet_add_rms_norm_bwd_workspace_bytes(10, 64)
    assert need > 0 and _norm_bwd(lib, wb=need - 1) == WS
    assert lib.deltanet_add_rms_norm_bwd_workspace_bytes(10, 60) == 0
    assert lib.deltanet_last_hip_error() == 0


def test_rows_of_none_launch_nothing(lib):
    assert _norm(lib, rows=0, x=None, y=None) == OK
    assert _conv(lib, L=0, x=None, y=None, s=None) == OK
    assert lib.deltanet_last_hip_error() == 0


def test_sizes_beyond_one_launch_are_refused(lib):
    assert _conv(lib, B=1, L=2 ** 30, D=2 ** 16) == UNSUP
    assert _scan(lib, B=2 ** 20, L=2 ** 20, D=2 ** 16) == UNSUP
    assert _scan_step(lib, B=2 ** 30, D=2 ** 20) == UNSUP
    assert _conv_step(lib, B=2 ** 31 - 1, D=2 ** 20) == UNSUP
    assert lib.deltanet_last_hip_error() == 0


def test_binding_refuses_wrong_tensors():
    x, w = torch.zeros(1, 4, 64), torch.zeros(64, 4)
    few, A = torch.zeros(1, 4, 16), torch.zeros(64, 16)
    with pytest.raises(ValueError, match="GPU"):
        binding.short_conv_fwd(x, w)
    with pytest.raises(ValueError, match="dimensions"):
        binding.short_conv_fwd(x[0], w)
    with pytest.raises(ValueError, match="dimensions"):
        binding.short_conv_step(x, w, None, x)
    with pytest.raises(ValueError, match="GPU"):
        binding.selective_scan_fwd(x, x, A, few, few)
    with pytest.raises(ValueError, match="dimensions"):
        binding.selective_scan_step(x, x, A, few, few, x)
    with pytest.raises(ValueError, match="GPU"):
        binding.add_rms_norm(x, None, None)
    with pytest.raises(ValueError, match="rows"):
        binding.add_rms_norm(torch.tensor(1.0), None, None)
    with pytest.raises(ValueError, match="batch must be 1"):
        binding._check_cu(torch.zeros(3, dtype=torch.int32), 2, x.device)
    with pytest.raises(ValueError, match=r"sequences \+ 1"):
        binding._check_cu(torch.zeros(1, dtype=torch.int32), 1, x.device)
