"""The state space layer's operators near the ends of what one launch takes (2^32 - 1 work-items)."""

import pytest
import torch

from deltanet_delta_rule_chunk_amd import binding as N
from ssm_cases import DEV, ULP

pytestmark = pytest.mark.gpu


def test_scan_gradient_of_many_channels(gpu_lib):
    """Two tokens of 7 million channels with 32 states (14.9 million workgroups add up dA):
    dA = C_2 g_2 e^{dt_2 A} (dt_1 u_1 B_1) dt_2, with |dt A| <= 4: 20 roundings of it are 2.5 x 4 of the
    exponent, 1 of the exponential and 9 of the products and the conversions."""
    D, S = 7_000_000, 32
    gen = torch.Generator(device=DEV).manual_seed(1)
    r = lambda *s: torch.randn(s, generator=gen, device=DEV)  # noqa: E731
    p = lambda *s: 0.5 + torch.rand(s, generator=gen, device=DEV)  # noqa: E731
    u, dt, dy, B, C = r(1, 2, D), p(1, 2, D), r(1, 2, D), r(1, 2, S), r(1, 2, S)
    A, skip = -p(D, S), r(D)
    dA, dD = (N.selective_scan_bwd(u, dt, A, B, C, dy, D=skip, softplus=False, want_dh0=False)[i] for i in (2, 5))
    for lo in range(0, D, 1_000_000):
        c = slice(lo, lo + 1_000_000)
        e = lambda t, i: t[0, i, c].double()  # noqa: E731
        want = (e(dy, 1) * e(dt, 0) * e(u, 0) * e(dt, 1))[:, None] * torch.exp(e(dt, 1)[:, None] * A[c].double())
        want *= C[0, 1].double() * B[0, 0].double()
        assert ((dA[c].double() - want).abs() <= 20 * ULP * want.abs() + 1e-37).all(), lo
        g = e(dy, 0) * e(u, 0), e(dy, 1) * e(u, 1)
        assert ((dD[c].double() - (g[0] + g[1])).abs() <= 3 * ULP * (g[0].abs() + g[1].abs())).all(), lo


@pytest.mark.parametrize("D,rows", [(8, 2 ** 26 + 3), (128, 2 ** 24 + 5), (264, 2 ** 24 + 5)])
def test_norm_of_many_rows(gpu_lib, D, rows):
    """More rows than a launch has workgroups: the last ones and the first are those of a call on their own."""
    gen = torch.Generator(device=DEV).manual_seed(2)
    r = lambda *s: torch.randn(s, generator=gen, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    x, res, w = r(rows, D), r(rows, D), torch.rand((D,), generator=gen, device=DEV)
    y, total = N.add_rms_norm(x, res, w)
    y8, scale, _ = N.add_rms_norm_fp8(x, res, w)
    d, _, dw = N.add_rms_norm_bwd(total, w, x, res)
    for s in (slice(0, 60), slice(rows // 2, rows // 2 + 60), slice(rows - 60, rows)):
        y1, t1 = N.add_rms_norm(x[s], res[s], w)
        q1, s1, _ = N.add_rms_norm_fp8(x[s], res[s], w)
        assert torch.equal(y[s], y1) and torch.equal(total[s], t1) and torch.equal(scale[s], s1)
        assert torch.equal(y8[s].view(torch.uint8), q1.view(torch.uint8))
        assert torch.equal(d[s], N.add_rms_norm_bwd(t1, w, x[s], res[s])[0])
    # dw in 64 bits: a group of lanes adds up one in 1024 x 4 (or 16) rows, a rounding each; 100 of the
    # terms besides, as in the norm's own tests.
    parts, size = torch.zeros(D, dtype=torch.float64, device=DEV), torch.zeros(D, dtype=torch.float64, device=DEV)
    for lo in range(0, rows, 2 ** 20):
        s = slice(lo, min(rows, lo + 2 ** 20))
        n = total[s].double()
        n = n / torch.sqrt((n * n).mean(-1, keepdim=True) + 1e-6)
        parts += (x[s].double() * n).sum(0)
        size += (x[s].double() * n).abs().sum(0)
    groups = 1024 * (16 if D <= 128 else 4)
    assert ((dw.double() - parts).abs() <= (100 + rows / groups + 1) * ULP * size).all()
