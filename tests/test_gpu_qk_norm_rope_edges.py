"""The differentiable norm with rotation: what its backward keeps and refuses."""

import pytest
import torch

from deltanet_delta_rule_chunk_amd import binding as N

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def _inputs():
    gen = torch.Generator(device=DEV).manual_seed(9)
    q = torch.randn((1, 3, 20, 64), generator=gen, device=DEV)
    k = torch.randn((1, 2, 20, 64), generator=gen, device=DEV)
    pos = torch.arange(40, device=DEV, dtype=torch.int32).view(2, 1, 20) * 7
    return q, k, pos, torch.rand(32, generator=gen, device=DEV)


def test_sections_changed_after_the_call(gpu_lib):
    q, k, pos, inv = _inputs()
    q.requires_grad_()
    sections = [8, 24]
    y, _ = N.rotary_qk(q, k, pos, inv, sections=sections)
    sections[:] = [24, 8]
    got, = torch.autograd.grad(y.sum(), q)
    y, _ = N.rotary_qk(q, k, pos, inv, sections=[8, 24])
    want, = torch.autograd.grad(y.sum(), q)
    assert torch.equal(got, want)


def test_a_frequency_that_asks_for_a_gradient_is_refused(gpu_lib):
    q, k, pos, inv = _inputs()
    inv.requires_grad_()
    with pytest.raises(ValueError, match="inv_freq"):
        N.rotary_qk(q, k, pos, inv, sections=[8, 24])
    with torch.no_grad():
        N.rotary_qk(q, k, pos, inv, sections=[8, 24])
    N.rotary_qk(q, k, pos, inv.detach(), sections=[8, 24])
