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
