"""Scales at the ends of bf16's range."""

import pytest
import torch

from expert_routed_ffn_gb300 import capi

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _built():
    from expert_routed_ffn_gb300 import build
    build.build()
    capi.load()
    yield
    assert capi.operators_status() == capi.MOE_OK


@pytest.mark.parametrize("steps", [1, 5])
@pytest.mark.parametrize("power", [-110, -100, -40, 0, 40, 120])
@pytest.mark.parametrize("N,K", [(64, 136), (264, 136)])
def test_a_power_of_two_scales_the_result_exactly(N, K, power, steps):
    """Results are at most 2, and bf16's normal numbers begin at 2^-126: down to 2^-16 of the unscaled ones they
    differ by the scale alone."""
    gen = torch.Generator(device="cuda").manual_seed(41)
    G = torch.randn(N, K, generator=gen, device="cuda")
    one = capi.orthogonalize(G, steps=steps).double()
    got = capi.orthogonalize(G, steps=steps, scale=2.0 ** power).double()
    large = one.abs() >= 2.0 ** -16
    assert float(large.double().mean()) > 0.99
    assert torch.equal(got[large], one[large] * 2.0 ** power)


@pytest.mark.parametrize("steps", [1, 5])
@pytest.mark.parametrize("scale", [1.47 * 2.0 ** -120, 1.47 * 2.0 ** -100, -1.47, 1.47 * 2.0 ** 125])
def test_any_scale_is_one_factor(steps, scale):
    """Both results are rounded once, by half a step of bf16 (2^-8) each; the factor's products by 2^-24."""
    gen = torch.Generator(device="cuda").manual_seed(42)
    G = torch.randn(40, 8, 8, generator=gen, device="cuda")
    one = capi.orthogonalize(G, steps=steps).double()
    got = capi.orthogonalize(G, steps=steps, scale=scale).double()
    large = one.abs() >= 2.0 ** -6  # 2^-126 after the smallest scale
    assert float(large.double().mean()) > 0.9
    assert bool(((got - scale * one).abs() <= (2.0 ** -7 + 2.0 ** -14) * (scale * one).abs())[large].all())
