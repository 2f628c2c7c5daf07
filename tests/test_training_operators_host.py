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


NORM = {"X": at(1), "F": at(2), "pre": at(3), "post": at(4), "gate": at(5), "gate_kind": 1, "alpha": 1.0, "eps": 1e-5, "kind": 1,
        "T": 16, "H": 64, "x_dtype": 0, "f_dtype": 0, "X_out": at(6), "N": at(7)}
NORM_BACKWARD = {"dX_out": at(1), "dN": at(2), "X_out": at(3), "F": at(4), "pre": at(5), "post": at(6), "gate": at(7), "gate_kind": 2,
                 "alpha": 1.0, "eps": 1e-5, "kind": 2, "T": 16, "H": 64, "x_dtype": 1, "f_dtype": 0, "dX": at(8), "dF": at(9),
                 "dpre": at(10), "dpost": at(11), "dgate": at(12), "work": at(13), "size": 1 << 20}


def norm(lib, **change):
    return lib.moe_sandwich_norm(*{**NORM, **change}.values(), None)


def norm_backward(lib, **change):
    return lib.moe_sandwich_norm_backward(*{**NORM_BACKWARD, **change}.values(), None)


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("call,base", [(norm, NORM), (norm_backward, NORM_BACKWARD)])
def test_norm_refusals(lib, call, base):
    for change, status in [({"T": -1}, INVALID), ({"H": 0}, INVALID), ({"H": 60}, UNSUPPORTED), ({"H": 8200}, UNSUPPORTED), ({"T": (1 << 30) + 1, "size": 1 << 40}, UNSUPPORTED),
                           ({"x_dtype": 2}, INVALID), ({"f_dtype": -1}, INVALID), ({"kind": 0}, INVALID), ({"kind": 3}, INVALID),
                           ({"gate_kind": 3}, INVALID), ({"gate_kind": 0}, INVALID), ({"gate": None}, INVALID),
                           ({"alpha": NAN}, INVALID), ({"alpha": INF}, INVALID), ({"eps": 0.0}, INVALID), ({"eps": NAN}, INVALID),
                           ({"eps": INF}, INVALID)] + [({k: ODD}, INVALID) for k, v in base.items() if isinstance(v, ctypes.c_void_p)]:
        assert call(lib, **{k: v for k, v in change.items() if k in base}) == status, change
        assert "moe_sandwich_norm" in lib.moe_last_error().decode()


def test_norm_parts_refusals(lib):
    for change in ({"X": None}, {"F": None}, {"X_out": None}, {"N": None}, {"pre": None},
                   {"F": None, "X_out": None},  # post_w and the gate are F's
                   {"F": None, "X_out": None, "post": None, "gate": None, "gate_kind": 0, "pre": None, "N": None}):
        assert norm(lib, **change) == INVALID, change
    for change in ({"dX": None}, {"F": None}, {"dF": None}, {"dN": None}, {"pre": None}, {"X_out": None}, {"work": None}, {"size": 16},
                   {"pre": None, "dN": None},  # dpre_w of no weight
                   {"post": None}, {"gate": None, "gate_kind": 0},
                   {"pre": None, "dN": None, "dpre": None, "dX_out": None}):
        assert norm_backward(lib, **change) == INVALID, change
    assert norm(lib, T=0) == OK and norm(lib, T=0, X=None, F=None, X_out=None, N=None, gate=None, gate_kind=0, post=None) == OK
    need = ctypes.c_size_t()
    assert lib.moe_sandwich_norm_workspace(-1, 64, ctypes.byref(need)) == INVALID
    assert lib.moe_sandwich_norm_workspace(4, 64, None) == INVALID
    assert lib.moe_sandwich_norm_workspace(4, 12, ctypes.byref(need)) == UNSUPPORTED
    assert lib.moe_sandwich_norm_workspace(4, 64, ctypes.byref(need)) == OK and need.value > 0


def test_norm_outputs_overlap(lib):
    in_place = {"X_out": "X", "N": "F", "dX": "dX_out", "dF": "dN"}
    for call, base, outs in ((norm, NORM, ["X_out", "N"]), (norm_backward, NORM_BACKWARD, ["dX", "dF", "dpre", "dpost", "dgate", "work"])):
        for out in outs:
            for other, value in base.items():
                if isinstance(value, ctypes.c_void_p) and other not in (out, in_place.get(out)):
                    assert call(lib, **{out: value}) == INVALID, (out, other)
            if out in in_place:  # in place, but shifted
                shifted = ctypes.c_void_p(base[in_place[out]].value + 16)
                assert call(lib, **{out: shifted}) == INVALID, out


QUINTIC = (3.4445, -4.7750, 2.0315)
ORTHO = {"G": at(1), "dtype": 1, "E": 2, "N": 64, "K": 128, "coefficients": QUINTIC * 5, "steps": 5, "eps": 1e-7, "scale": 1.0,
         "out": at(2), "work": at(3), "size": 1 << 22}


def ortho(lib, **change):
    a = {**ORTHO, **change}
    if a["coefficients"] is not None:
        a["coefficients"] = (ctypes.c_float * len(a["coefficients"]))(*a["coefficients"])
    return lib.moe_orthogonalize(*a.values(), None)


def test_orthogonalize_refusals(lib):
    for change, status in [({"G": None}, INVALID), ({"out": None}, INVALID), ({"work": None}, INVALID), ({"G": ODD}, INVALID),
                           ({"out": ODD}, INVALID), ({"work": ODD}, INVALID), ({"dtype": 2}, INVALID), ({"E": -1}, INVALID),
                           ({"N": 0}, INVALID), ({"K": -8}, INVALID), ({"N": 60}, UNSUPPORTED), ({"K": 16392}, UNSUPPORTED),
                           ({"E": 65536}, UNSUPPORTED), ({"steps": 0}, INVALID), ({"steps": 65, "coefficients": QUINTIC * 65}, INVALID),
                           ({"coefficients": None}, INVALID), ({"coefficients": QUINTIC * 4 + (NAN, 0.0, 0.0)}, INVALID),
                           ({"coefficients": QUINTIC * 4 + (INF, 0.0, 0.0)}, INVALID), ({"coefficients": (40.0, 0.0, 0.0) * 5}, UNSUPPORTED),
                           ({"eps": 0.0}, INVALID), ({"eps": NAN}, INVALID), ({"scale": NAN}, INVALID), ({"size": 1024}, INVALID),
                           ({"out": at(1)}, INVALID), ({"work": at(1)}, INVALID), ({"work": at(2)}, INVALID),
                           ({"out": ctypes.c_void_p((1 << 24) + 16), "dtype": 0}, INVALID)]:
        assert ortho(lib, **change) == status, change
        assert "moe_orthogonalize" in lib.moe_last_error().decode()
    assert ortho(lib, E=0, G=None, out=None, work=None, size=0) == OK
    need = ctypes.c_size_t()
    assert lib.moe_orthogonalize_workspace(2, 64, 128, None) == INVALID
    assert lib.moe_orthogonalize_workspace(2, 64, 100, ctypes.byref(need)) == UNSUPPORTED
    assert lib.moe_orthogonalize_workspace(2, 64, 128, ctypes.byref(need)) == OK and need.value <= ORTHO["size"]
