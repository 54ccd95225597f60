"""The short convolution where there are rows enough for its longest runs, and the norm's
gradient where a group of lanes takes several rows, in the forms that smaller calls do not
reach.

Rows of the convolution depend on K - 1 neighbours alone and their arithmetic is the same in
every run, so a whole call's rows are those of calls on parts of them, to the bit.  Its weights'
gradient: 30 fp32 roundings as in the convolution's own tests, 64 of a run's rows, 3 of the four
waves' sums and one of the result, of the terms' magnitudes, which are formed here in 64 bits on the
GPU.  The norm's bounds are those of its own tests.
"""

import numpy as np
import pytest
import torch

from deltanet_delta_rule_chunk_amd import binding as N
from oracle import add_norm_backward
from ssm_cases import DEV, TYPES, ULP, close, cu_of, f64, normal

pytestmark = pytest.mark.gpu


def _inputs(seed, L, D, K, dtype, n):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    r = lambda *s, t=torch.float32: torch.randn(s, generator=gen, device=DEV).to(t)  # noqa: E731
    t = TYPES[dtype]
    return r(1, L, D, t=t), r(D, K) * K ** -0.5, r(D), r(n, K - 1, D, t=t), r(1, L, D, t=t), r(n, K - 1, D, t=t)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("K", [2, 3, 4])
def test_long_runs_are_their_parts(gpu_lib, dtype, K):
    L, D = 33000, 4096
    cuts = [3, 3, 5000, 5001, 20007, 32990]
    x, w, b, s0, dy, ds = _inputs(K, L, D, K, dtype, 5)
    y, s = N.short_conv_fwd(x, w, b, s0, cu_seqlens=cu_of(cuts))
    dx, dw, db, ds0 = N.short_conv_bwd(x, w, b, s0, dy, ds, cu_seqlens=cu_of(cuts))
    for t in (y, dx):
        assert not t[:, :3].any() and not t[:, 32990:].any()
    for i, (lo, hi) in enumerate(zip(cuts[:-1], cuts[1:])):
        if hi == lo:
            assert torch.equal(s[i], s0[i]) and torch.equal(ds0[i], ds[i])
            continue
        for at, end in ((lo, min(hi, lo + 400)), (max(lo, hi - 400), hi)):
            # (From 3 rows before: their taps reach them, and their gradients those behind them.)
            front = s0[i:i + 1] if at - lo < K - 1 else x[:, at - (K - 1):at].contiguous()
            if 0 < at - lo < K - 1:
                continue
            back = None if end < hi else ds[i:i + 1]
            part = (x[:, at:end].contiguous(), w, b, front)
            y1, s1 = N.short_conv_fwd(*part)
            assert torch.equal(y[:, at:end], y1)
            dx1, _, _, ds1 = N.short_conv_bwd(*part, dy[:, at:end].contiguous(), back)
            keep = end - at if end == hi else end - at - (K - 1)
            assert torch.equal(dx[:, at:at + keep], dx1[:, :keep])
            if end == hi:
                assert torch.equal(s[i], s1[0])
            if at == lo:
                assert torch.equal(ds0[i], ds1[0])
    # The weights' gradient, 512 channels at a time.
    for c in range(0, D, 512):
        d = slice(c, c + 512)
        want, size = torch.zeros((512, K + 1), device=DEV, dtype=torch.float64), torch.zeros((512, K + 1), device=DEV, dtype=torch.float64)
        for i, (lo, hi) in enumerate(zip(cuts[:-1], cuts[1:])):
            e = torch.cat([s0[i, :, d], x[0, lo:hi, d]]).double()
            n = hi - lo
            p = sum(w[d, j].double() * e[j:j + n] for j in range(K)) + b[d].double()
            pm = sum(w[d, j].double().abs() * e[j:j + n].abs() for j in range(K)) + b[d].double().abs()
            g = torch.sigmoid(p)
            q = dy[0, lo:hi, d].double() * g * (1 + p * (1 - g))
            qm = dy[0, lo:hi, d].double().abs() * (1.1 + 0.5 * pm)
            for j in range(K):
                want[:, j] += (q * e[j:j + n]).sum(0)
                size[:, j] += (qm * e[j:j + n].abs()).sum(0)
            want[:, K] += q.sum(0)
            size[:, K] += qm.sum(0)
        got = torch.cat([dw[d], db[d, None]], 1).double()
        assert ((got - want).abs() <= (30 + 64 + 4) * ULP * size).all()


@pytest.mark.parametrize("dtype,wide", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("rows,D", [(20000, 8), (17001, 128), (9000, 136), (3001, 4096), (700, 16392), (600, 32768)])
def test_norm_gradient_of_several_rows_per_group(gpu_lib, dtype, wide, rows, D):
    gen = torch.Generator().manual_seed(D)
    t, r = TYPES[dtype], TYPES[wide]
    total, w = normal(gen, (rows, D), 2.0, dtype=r), 1 + normal(gen, (D,), 0.3)
    dy, dt = normal(gen, (rows, D), dtype=t), normal(gen, (rows, D), dtype=r)
    dx, dr, dw = N.add_rms_norm_bwd(*(v.to(DEV) for v in (total, w, dy, dt)))
    e, ew = f64(total), f64(w)
    d, dwe = add_norm_backward(e, ew, f64(dy), f64(dt), 1e-6)
    root = 1 / np.sqrt((e ** 2).mean(-1, keepdims=True) + 1e-6)
    n, g = np.abs(e * root), np.abs(f64(dy) * ew)
    size = np.abs(f64(dt)) + root * (g + n * (n * g).mean(-1, keepdims=True))
    close(dx, d, size, 100, "dx")
    close(dr, d, size, 100, "dresidual")
    close(dw, dwe, (np.abs(f64(dy)) * n).sum(0), 100 + rows, "dweight")
