"""The operators' argument checks, before anything touches a device (no GPU needed)."""

import ctypes

import pytest

from expert_routed_ffn_gb300 import build as moe_build
from expert_routed_ffn_gb300 import capi

FAKE = ctypes.c_void_p(1 << 20)  # aligned, never dereferenced: validation fails first
ODD = ctypes.c_void_p((1 << 20) + 8)


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return capi.load()


GROUPED = {"a": FAKE, "b": FAKE, "offs": FAKE, "rows": 16, "E": 4, "N": 64, "K": 64, "out_dtype": 0, "out": FAKE}


@pytest.mark.parametrize("change,status", [
    ({"rows": -1}, capi.MOE_ERR_INVALID_ARG), ({"E": 0}, capi.MOE_ERR_INVALID_ARG), ({"N": 0}, capi.MOE_ERR_INVALID_ARG),
    ({"K": -8}, capi.MOE_ERR_INVALID_ARG), ({"out_dtype": 2}, capi.MOE_ERR_INVALID_ARG), ({"a": None}, capi.MOE_ERR_INVALID_ARG),
    ({"b": None}, capi.MOE_ERR_INVALID_ARG), ({"offs": None}, capi.MOE_ERR_INVALID_ARG), ({"out": None}, capi.MOE_ERR_INVALID_ARG),
    ({"a": ODD}, capi.MOE_ERR_INVALID_ARG), ({"b": ODD}, capi.MOE_ERR_INVALID_ARG), ({"out": ODD}, capi.MOE_ERR_INVALID_ARG),
    ({"offs": ctypes.c_void_p((1 << 20) + 2)}, capi.MOE_ERR_INVALID_ARG), ({"E": 257}, capi.MOE_ERR_UNSUPPORTED),
    ({"N": 60}, capi.MOE_ERR_UNSUPPORTED), ({"K": 100}, capi.MOE_ERR_UNSUPPORTED), ({"N": (1 << 20) + 8}, capi.MOE_ERR_UNSUPPORTED),
    ({"rows": (1 << 30) + 1}, capi.MOE_ERR_UNSUPPORTED),
])
@pytest.mark.parametrize("op", ["forward", "dgrad", "wgrad"])
def test_grouped_refusals(lib, op, change, status):
    a = {**GROUPED, **change}
    head = [a[k] for k in ("a", "b", "offs", "rows", "E", "N", "K", "out_dtype")] + ([0] if op == "wgrad" else [])
    assert getattr(lib, f"moe_grouped_{op}")(*head, a["out"], None) == status
    assert f"moe_grouped_{op}" in lib.moe_last_error().decode()


def test_grouped_special_arguments(lib):
    assert lib.moe_grouped_forward(None, None, None, 0, 4, 64, 64, 0, None, None) == capi.MOE_OK  # no rows: nothing to do
    assert lib.moe_grouped_dgrad(None, None, None, 0, 4, 64, 64, 0, None, None) == capi.MOE_OK
    assert lib.moe_grouped_wgrad(FAKE, FAKE, FAKE, 16, 4, 64, 64, 0, 2, FAKE, None) == capi.MOE_ERR_INVALID_ARG
    assert lib.moe_grouped_wgrad(None, None, None, 0, 4, 64, 64, 0, 0, None, None) == capi.MOE_ERR_INVALID_ARG
    assert lib.moe_grouped_wgrad(None, None, None, 0, 4, 64, 64, 0, 1, FAKE, None) == capi.MOE_OK
