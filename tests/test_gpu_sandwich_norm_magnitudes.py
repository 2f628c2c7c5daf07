"""Rows of F near the end of fp32's range, whose norm's inverse is at or under the least normal number, with
gates that make it smaller still.  Bounds as in tests/test_gpu_sandwich_norm.py."""

import pytest
import torch

from expert_routed_ffn_gb300 import capi
from tests.test_gpu_sandwich_norm import BF, F32, _check_backward, _check_forward, _inputs

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_routed_ffn_gb300 import build
    build.build()
    capi.load()


@pytest.fixture(autouse=True)
def _status():
    yield
    assert capi.operators_status() == capi.MOE_OK


@pytest.mark.parametrize("gate", ["token", "channel"])
@pytest.mark.parametrize("small", [1.0, 1e-5, 1e-9])
@pytest.mark.parametrize("types", [(F32, F32), (F32, BF), (BF, BF)])
@pytest.mark.parametrize("T,H", [(37, 200), (64, 520), (5, 8192)])
def test_gates_on_rows_of_largest_values(T, H, types, small, gate):
    s = _inputs(T, H, *types, gate, "rms", seed=23)
    s["F"] = (s["F"].float() * 8e36).to(types[1])  # 3 standard deviations of 2.4e37: up to 1.3e38
    s["gate"] = s["gate"] * small
    s["X"] = (s["X"].float() * small).to(types[0])  # beside which the gated block still counts
    s["dX"] = (s["dX"].float() * 1e20).to(types[0])  # so that the gradient of F is a normal number
    assert bool(torch.isfinite(s["F"]).all())
    how = dict(pre_w=s["pre_w"], post_w=s["post_w"], gate=s["gate"], residual_scale=0.5, eps=1e-5, kind="rms")
    _check_forward(capi.sandwich_norm(s["X"], s["F"], **how), s, "rms", 0.5, 1e-5)
    _check_backward(capi.sandwich_norm_backward(s["dX"], s["dN"], s["X"], s["F"], **how), s, "rms", 0.5, 1e-5)
