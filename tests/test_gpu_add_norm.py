"""The norm with the residual's addition against fp64.

Bounds, in fp32 roundings: the sum of squares one per addition along a lane's pieces and
its shuffles (at most 32 + 10, halved by the root), 4 for the root, the quotient and the products: 40
covers every row length.  The gradient has two such sums: 100 of |dtotal| + r (|v| +
|n| mean |n v|); its weights one per row of a workgroup besides.
"""

import numpy as np
import pytest
import torch

from deltanet_delta_rule_chunk_amd import binding as N
from oracle import add_norm, add_norm_backward
from ssm_cases import DEV, TYPES, close, f64, normal

pytestmark = pytest.mark.gpu
#: One of every group of lanes and pieces, and odd ones between.
WIDTHS = [8, 128, 136, 504, 520, 1024, 1032, 2048, 2072, 4096, 4104, 8192, 8200, 16384, 16392, 32768]
PAIRS = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")]


def _inputs(seed, rows, D, dtype, wide):
    gen = torch.Generator().manual_seed(seed)
    t, r = TYPES[dtype], TYPES[wide]
    x, res = normal(gen, (rows, D), dtype=t), normal(gen, (rows, D), 2.0, dtype=r)
    return x, res, 1 + normal(gen, (D,), 0.3), normal(gen, (rows, D), dtype=t), normal(gen, (rows, D), dtype=r)


@pytest.mark.parametrize("dtype,wide", PAIRS)
@pytest.mark.parametrize("D", WIDTHS)
def test_forward_and_backward(gpu_lib, dtype, wide, D):
    rows, eps = 37, 1e-5
    x, res, w, dy, dt = _inputs(D, rows, D, dtype, wide)
    y, total = N.add_rms_norm(x.to(DEV), res.to(DEV), w.to(DEV), eps=eps)
    want = (x.double() + res.double()).to(res.dtype)
    assert torch.equal(total.cpu(), want)  # (the sum of two bf16, or of fp32, rounded once)
    e, ew = f64(want), f64(w)
    v = add_norm(e, ew, eps)
    close(y, v, np.abs(v), 40, "y")
    dx, dr, dw = N.add_rms_norm_bwd(total, w.to(DEV), dy.to(DEV), dt.to(DEV), eps=eps)
    d, dwe = add_norm_backward(e, ew, f64(dy), f64(dt), eps)
    r = 1 / np.sqrt((e ** 2).mean(-1, keepdims=True) + eps)
    n, g = np.abs(e * r), np.abs(f64(dy) * ew)
    size = np.abs(f64(dt)) + r * (g + n * (n * g).mean(-1, keepdims=True))
    close(dx, d, size, 100, "dx")
    close(dr, d, size, 100, "dresidual")
    assert (dr is dx) == (dtype == wide)
    close(dw, dwe, (np.abs(f64(dy)) * n).sum(0), 100 + rows, "dweight")


@pytest.mark.parametrize("rows", [1, 3, 1023, 5000])
def test_many_rows(gpu_lib, rows):
    x, res, w, dy, dt = (t.to(DEV) for t in _inputs(rows, rows, 264, "bf16", "bf16"))
    y, total = N.add_rms_norm(x, res, w)
    dx, _, dw = N.add_rms_norm_bwd(total, w, dy, dt)
    e, ew = f64(total), f64(w)
    v = add_norm(e, ew, 1e-6)
    close(y, v, np.abs(v), 40, "y")
    _, dwe = add_norm_backward(e, ew, f64(dy), f64(dt), 1e-6)
    r = 1 / np.sqrt((e ** 2).mean(-1, keepdims=True) + 1e-6)
    close(dw, dwe, (np.abs(f64(dy)) * np.abs(e * r)).sum(0), 100 + rows, "dweight")


@pytest.mark.parametrize("dtype,wide", PAIRS)
@pytest.mark.parametrize("D", [8, 136, 1032, 2072, 4096, 8200, 20480])
def test_8_bits(gpu_lib, dtype, wide, D):
    x, res, w, _, _ = _inputs(D + 1, 19, D, dtype, wide)
    res[3], x[3] = 0.0, 0.0                      # a row of zeros
    y8, scale, total = N.add_rms_norm_fp8(x.to(DEV), res.to(DEV), w.to(DEV))
    assert y8.dtype == torch.float8_e4m3fn and scale.shape == (19,) and float(scale[3]) == 1.0
    v = add_norm(f64(total), f64(w), 1e-6)
    top = np.abs(v).max(-1)
    s = f64(scale)
    live = np.arange(19) != 3
    assert (np.abs(s[live] * 448 - top[live]) <= 45 * 2.0 ** -24 * top[live]).all()
    got = f64(y8.float()) * s[:, None]
    # Half a step of e4m3: 2^-4 of the value, or 2^-10 (its smallest step is 2^-9) times the scale.
    half = np.maximum(np.abs(v) * 2.0 ** -4, s[:, None] * 2.0 ** -10)
    assert (np.abs(got - v) <= half * (1 + 100 * 2.0 ** -24) + 100 * 2.0 ** -24 * np.abs(v)).all()
    assert f64(y8.float())[live].__abs__().max(-1).min() == 448.0
    # The values are those of the quotients in 64 bits.
    vw = f64(total) * f64(w)
    q = torch.from_numpy(vw[live] * (448 / np.abs(vw[live]).max(-1, keepdims=True))).float().to(torch.float8_e4m3fn)
    assert torch.equal(q.view(torch.uint8), y8.cpu()[torch.from_numpy(live)].view(torch.uint8))


@pytest.mark.parametrize("size,weight", [(1.0, 2.0 ** -100), (2.0 ** 30, 2.0 ** 100), (2.0 ** -60, 1.0), (2.0 ** 55, 1.0)])
def test_8_bits_of_small_and_large(gpu_lib, size, weight):
    # (264 squares of 2^60 times a normal number pass 2^128, where the row overflows: 2^55 stays within.)
    x, _, w, _, _ = _inputs(3, 7, 264, "f32", "f32")
    x, w = x.double() * size, w.double() * weight   # (scaled by powers of two: exact in fp32)
    y8, scale, _ = N.add_rms_norm_fp8(x.float().to(DEV), None, w.float().to(DEV), eps=0.0)
    v = add_norm(f64(x), f64(w), 0.0)
    top = np.abs(v).max(-1)
    assert (np.abs(f64(scale) * 448 - top) <= 45 * 2.0 ** -24 * top).all()
    vw = f64(x) * f64(w)
    q = torch.from_numpy(vw * (448 / np.abs(vw).max(-1, keepdims=True))).float().to(torch.float8_e4m3fn)
    assert torch.equal(q.view(torch.uint8), y8.cpu().view(torch.uint8))


def test_8_bits_where_a_row_overflows_and_weights_that_are_not_finite(gpu_lib):
    x, _, w, _, _ = (t.to(DEV) for t in _inputs(4, 5, 264, "f32", "f32"))
    x[2] *= 2.0 ** 80
    y8, scale, _ = N.add_rms_norm_fp8(x, None, w)
    assert float(scale[2]) == 1.0 and not y8[2].float().any() and y8[1].float().any()
    for bad in (float("nan"), float("inf")):
        w[9] = bad
        y8, scale, _ = N.add_rms_norm_fp8(x, None, w)
        assert scale.isnan().all() and y8.float().isnan().all()


def test_without_residual_weight_and_in_place(gpu_lib):
    x, res, w, dy, dt = (t.to(DEV) for t in _inputs(5, 11, 264, "bf16", "bf16"))
    y, total = N.add_rms_norm(x, None, None)
    assert total is x
    v = add_norm(f64(x), np.ones(264), 1e-6)
    close(y, v, np.abs(v), 40, "y")
    dx, _, dw = N.add_rms_norm_bwd(x, None, dy)
    d, _ = add_norm_backward(f64(x), np.ones(264), f64(dy), None, 1e-6)
    r = 1 / np.sqrt((f64(x) ** 2).mean(-1, keepdims=True) + 1e-6)
    n, g = np.abs(f64(x) * r), np.abs(f64(dy))
    close(dx, d, r * (g + n * (n * g).mean(-1, keepdims=True)), 100, "dx")
    assert dw is None
    want = N.add_rms_norm(x, res, w)
    stream = res.clone()
    got = N.add_rms_norm(x, stream, w, total=stream)
    assert got[1] is stream and torch.equal(stream, want[1]) and torch.equal(got[0], want[0])
    first = x.clone()
    got = N.add_rms_norm(first, res, w, total=first)
    assert torch.equal(first, want[1]) and torch.equal(got[0], want[0])


def test_shapes(gpu_lib):
    x, res, w, dy, _ = (t.to(DEV) for t in _inputs(6, 12, 64, "bf16", "bf16"))
    y, total = N.add_rms_norm(x, res, w)
    y3, t3 = N.add_rms_norm(x.view(3, 4, 64), res.view(3, 4, 64), w)
    assert torch.equal(y3.view(12, 64), y) and torch.equal(t3.view(12, 64), total)
    assert N.add_rms_norm_fp8(x.view(3, 4, 64), None, w)[1].shape == (3, 4)
    y1, t1 = N.add_rms_norm(x[0], res[0], w)
    assert torch.equal(y1, y[0]) and torch.equal(t1, total[0])
    y0, t0 = N.add_rms_norm(x[:0], res[:0], w)
    assert y0.shape == (0, 64) and t0.shape == (0, 64)
    dx, _, dw = N.add_rms_norm_bwd(t0, w, dy[:0])
    assert dx.shape == (0, 64) and not dw.any()


def test_what_is_not_finite_stays_in_its_row(gpu_lib):
    for D in (64, 264, 4096):
        x, res, w, dy, dt = (t.to(DEV) for t in _inputs(7, 9, D, "bf16", "bf16"))
        want = (*N.add_rms_norm(x, res, w), *N.add_rms_norm_fp8(x, res, w)[:2])
        x[4, 7], x[5, 3] = float("nan"), float("inf")
        got = (*N.add_rms_norm(x, res, w), *N.add_rms_norm_fp8(x, res, w)[:2])
        keep = [0, 1, 2, 3, 6, 7, 8]
        for a, b in zip(want, got):
            a, b = (t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t for t in (a, b))
            assert torch.equal(a[keep], b[keep])
        assert got[0][4].isnan().all() and got[3][4].isnan() and got[2][4].float().isnan().all()
        d = N.add_rms_norm_bwd(got[1], w, dy, dt)[0]
        assert d[4].isnan().all() and torch.isfinite(d[keep]).all()


def test_autograd(gpu_lib):
    for dtype, wide in PAIRS:
        x, res, w, dy, dt = (t.to(DEV) for t in _inputs(8, 10, 136, dtype, wide))
        leaves = [x.requires_grad_(), res.requires_grad_(), w.requires_grad_()]
        y, total = N.residual_norm(*leaves)
        d = torch.autograd.grad([y, total], leaves, [dy, dt])
        with torch.no_grad():
            want = N.add_rms_norm_bwd(total.detach(), w, dy, dt)
        for a, b in zip(d, want):
            assert torch.equal(a, b)
        y, same = N.residual_norm(leaves[0], None, leaves[2])
        assert same is leaves[0]
        d = torch.autograd.grad(y, [leaves[0], leaves[2]], dy)
        with torch.no_grad():
            want = N.add_rms_norm_bwd(x.detach(), w, dy)
        assert torch.equal(d[0], want[0]) and torch.equal(d[1], want[2])


def test_refusals(gpu_lib):
    x = torch.zeros((4, 64), device=DEV)
    with pytest.raises(ValueError, match="weight has shape"):
        N.add_rms_norm(x, None, torch.zeros(65, device=DEV))
    with pytest.raises(ValueError, match="residual has shape"):
        N.add_rms_norm(x, x[:3], None)
    with pytest.raises(ValueError, match="contiguous"):
        N.add_rms_norm(torch.zeros((64, 4), device=DEV).t(), None, None)
    with pytest.raises(ValueError, match="only written with a residual"):
        N.add_rms_norm(x, None, None, total=x)
    with pytest.raises(N.DeltaNetError, match="UNSUPPORTED"):
        N.add_rms_norm(x, x.bfloat16(), None)      # a narrower stream than x
    with pytest.raises(N.DeltaNetError, match="UNSUPPORTED"):
        N.add_rms_norm(torch.zeros((4, 32776), device=DEV), None, None)
    with pytest.raises(N.DeltaNetError, match="ALIASING"):
        N.add_rms_norm(x, None, None, y=x)
    with pytest.raises(TypeError, match="dtype"):
        N.add_rms_norm(x.half(), None, None)


def test_smallest_rows_in_8_bits(gpu_lib):
    """Rows whose scale would be below fp32's normal numbers: quotients stay numbers."""
    x = torch.zeros((3, 64), device=DEV)
    x[0, 1], x[1, 2], x[2] = 1e-38, 1e-42, 3e-39
    y8, scale, _ = N.add_rms_norm_fp8(x, None, None, eps=1.0)
    y = y8.float() * scale[:, None]
    assert torch.isfinite(y8.float()).all() and (scale >= 2.0 ** -126).all()
    # Half of the smallest step of e4m3, 2^-10, of the scale (sums of squares underflow: r = 1).
    assert float((y - x).abs().max()) <= 2.0 ** -10 * float(scale.max()) + 2.0 ** -4 * 1e-38
