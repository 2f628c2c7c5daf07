"""The argument checks of the operators that train an expert layer, before anything touches a device
(no GPU needed)."""

import ctypes

import pytest

from expert_routed_ffn_gb300 import build as moe_build
from expert_routed_ffn_gb300 import capi

INVALID, UNSUPPORTED, OK = capi.MOE_ERR_INVALID_ARG, capi.MOE_ERR_UNSUPPORTED, capi.MOE_OK


def at(n):
    """An address that is never dereferenced: validation fails first."""
    return ctypes.c_void_p(n << 24)


ODD = ctypes.c_void_p((1 << 24) + 8)


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return capi.load()


SIZES = {"rows": 16, "E": 4, "I": 64, "K": 64}
ACT = {"act": 1, "alpha": 1.7, "limit": 7.0, "beta": 1.0}
GATED = {
    "forward": {"X": at(1), "Wg": at(2), "Wu": at(3), "offs": at(4), **SIZES, **ACT, "H": at(5), "G": at(6), "U": at(7)},
    "backward": {"dY": at(1), "Wd": at(2), "G": at(3), "U": at(4), "offs": at(5), **SIZES, **ACT, "dG": at(6), "dU": at(7)},
    "dgrad": {"dG": at(1), "dU": at(2), "Wg": at(3), "Wu": at(4), "offs": at(5), **SIZES, "out_dtype": 0, "dX": at(6)},
}


def gated(lib, op, **change):
    args = {**GATED[op], **change}
    assert args.keys() == GATED[op].keys()
    return getattr(lib, f"moe_grouped_gated_{op}")(*args.values(), None)


@pytest.mark.parametrize("op", list(GATED))
def test_gated_refusals(lib, op):
    pointers = [k for k, v in GATED[op].items() if isinstance(v, ctypes.c_void_p)]
    for change, status in [({"rows": -1}, INVALID), ({"E": 0}, INVALID), ({"I": 0}, INVALID), ({"K": -8}, INVALID),
                           ({"E": 257}, UNSUPPORTED), ({"I": 60}, UNSUPPORTED), ({"K": 100}, UNSUPPORTED),
                           ({"I": (1 << 20) + 8}, UNSUPPORTED), ({"rows": (1 << 30) + 1}, UNSUPPORTED)] + \
            [({p: None}, INVALID) for p in pointers] + [({p: ODD}, INVALID) for p in pointers if p != "offs"] + \
            [({"offs": ctypes.c_void_p((1 << 24) + 2)}, INVALID)]:
        assert gated(lib, op, **change) == status, change
        assert f"moe_grouped_gated_{op}" in lib.moe_last_error().decode()
    assert gated(lib, op, rows=0, **{p: None for p in pointers}) == OK  # nothing to do


@pytest.mark.parametrize("op", ["forward", "backward"])
def test_gated_activation_refusals(lib, op):
    nan, inf = float("nan"), float("inf")
    for change in ({"act": 2}, {"act": -1}, {"limit": 0.0}, {"limit": -1.0}, {"limit": nan}, {"alpha": nan}, {"alpha": inf},
                   {"beta": nan}, {"beta": -inf}):
        assert gated(lib, op, **change) == INVALID, change


def test_gated_outputs_overlap(lib):
    for op, outs in (("forward", "HGU"), ("backward", ["dG", "dU"]), ("dgrad", ["dX"])):
        for out in outs:
            for other, value in GATED[op].items():
                if isinstance(value, ctypes.c_void_p) and other != out:
                    assert gated(lib, op, **{out: value}) == INVALID, (op, out, other)
    inside = ctypes.c_void_p((1 << 24) + 16 * 64 * 2 - 16)  # the last bytes of X
    assert gated(lib, "forward", H=inside) == INVALID
    assert gated(lib, "dgrad", dX=inside) == INVALID
    assert gated(lib, "dgrad", out_dtype=2) == INVALID
