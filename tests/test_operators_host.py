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


QUANT = {"X": FAKE, "dtype": 0, "slices": 2, "rows": 16, "K": 64, "format": 2, "codes": FAKE, "scales": FAKE}


@pytest.mark.parametrize("change,status", [
    ({"X": None}, capi.MOE_ERR_INVALID_ARG), ({"codes": None}, capi.MOE_ERR_INVALID_ARG), ({"scales": None}, capi.MOE_ERR_INVALID_ARG),
    ({"X": ODD}, capi.MOE_ERR_INVALID_ARG), ({"codes": ODD}, capi.MOE_ERR_INVALID_ARG), ({"scales": ODD}, capi.MOE_ERR_INVALID_ARG),
    ({"dtype": 2}, capi.MOE_ERR_INVALID_ARG), ({"slices": -1}, capi.MOE_ERR_INVALID_ARG), ({"rows": -1}, capi.MOE_ERR_INVALID_ARG),
    ({"K": 0}, capi.MOE_ERR_INVALID_ARG), ({"K": 48}, capi.MOE_ERR_UNSUPPORTED), ({"format": 0}, capi.MOE_ERR_INVALID_ARG),
    ({"format": 3}, capi.MOE_ERR_INVALID_ARG), ({"slices": 1 << 30, "rows": 1 << 30}, capi.MOE_ERR_UNSUPPORTED),
    ({"rows": 0, "X": None}, capi.MOE_OK), ({"slices": 0, "codes": None}, capi.MOE_OK),
])
def test_mx_refusals(lib, change, status):
    a = {**QUANT, **change}
    assert lib.moe_mx_quantize(*[a[k] for k in ("X", "dtype", "slices", "rows", "K", "format", "codes", "scales")], None) == status
    assert lib.moe_mx_dequantize(*[a[k] for k in ("codes", "scales", "format", "slices", "rows", "K", "dtype", "X")], None) == status


def test_clip_refusals(lib):
    need = ctypes.c_size_t()
    assert lib.moe_clip_workspace(-1, ctypes.byref(need)) == capi.MOE_ERR_INVALID_ARG
    assert lib.moe_clip_workspace(3, None) == capi.MOE_ERR_INVALID_ARG
    assert lib.moe_clip_workspace(3, ctypes.byref(need)) == capi.MOE_OK and need.value > 0

    def call(grad=FAKE, out=FAKE, count=8, dtype=1, n=1, max_norm=1.0, norm=FAKE, work=FAKE, size=need.value, table=True):
        t = (capi.MoeGrad * 1)(capi.MoeGrad(grad, out, count, dtype))
        return lib.moe_clip_grad_norm(t if table else None, n, max_norm, norm, work, size, None)

    for bad in (dict(grad=None), dict(out=None), dict(count=-1), dict(dtype=2), dict(n=-1), dict(max_norm=0.0),
                dict(max_norm=float("nan")), dict(norm=None), dict(work=None), dict(size=need.value - 1), dict(table=False),
                dict(work=ODD), dict(grad=ctypes.c_void_p((1 << 20) + 2)), dict(out=ctypes.c_void_p((1 << 20) + 1), dtype=0),
                dict(norm=ctypes.c_void_p((1 << 20) + 2))):
        assert call(**bad) == capi.MOE_ERR_INVALID_ARG, bad
        assert "moe_clip_grad_norm" in lib.moe_last_error().decode()


MX_GROUPED = {"Xc": FAKE, "Xs": FAKE, "Wc": FAKE, "Ws": FAKE, "offs": FAKE, "rows": 16, "E": 4, "N": 64, "K": 64, "out_dtype": 0,
              "Y": FAKE}


@pytest.mark.parametrize("change,status", [
    *[({k: None}, capi.MOE_ERR_INVALID_ARG) for k in ("Xc", "Xs", "Wc", "Ws", "offs", "Y")],
    *[({k: ODD}, capi.MOE_ERR_INVALID_ARG) for k in ("Xc", "Xs", "Wc", "Ws", "Y")],
    ({"rows": -1}, capi.MOE_ERR_INVALID_ARG), ({"E": 0}, capi.MOE_ERR_INVALID_ARG), ({"out_dtype": -1}, capi.MOE_ERR_INVALID_ARG),
    ({"E": 257}, capi.MOE_ERR_UNSUPPORTED), ({"N": 60}, capi.MOE_ERR_UNSUPPORTED), ({"K": 48}, capi.MOE_ERR_UNSUPPORTED),
    ({"rows": 0, "Xc": None, "Y": None}, capi.MOE_OK),
])
def test_mx_grouped_refusals(lib, change, status):
    a = {**MX_GROUPED, **change}
    assert lib.moe_mx_grouped_forward(*a.values(), None) == status


def test_wait_limit_refuses_what_is_no_bound(lib):
    assert lib.moe_operators_wait_limit(-2) == capi.MOE_ERR_INVALID_ARG
    assert lib.moe_operators_wait_limit(-1) == capi.MOE_OK


def _at(byte):
    return ctypes.c_void_p((1 << 30) + byte)


def test_outputs_that_overlap_inputs_are_refused(lib):
    """16 rows, E 4, N = K = 64, bf16: rows are 2 KB, the weights 32 KB; the offsets 20 bytes."""
    far, offs = _at(1 << 20), _at(1 << 21)
    for op, sizes in (("forward", (2048, 32768, 2048)), ("dgrad", (2048, 32768, 2048)), ("wgrad", (2048, 2048, 32768))):
        tail = [0] if op == "wgrad" else []
        for a, b, o, out in ((_at(0), far, offs, _at(sizes[0] - 16)), (far, _at(0), offs, _at(sizes[1] - 16)),
                             (_at(sizes[2] - 16), far, offs, _at(0)), (far, _at(1 << 22), _at(16), _at(0))):
            args = [a, b, o, 16, 4, 64, 64, 0, *tail, out, None]
            assert getattr(lib, f"moe_grouped_{op}")(*args) == capi.MOE_ERR_INVALID_ARG
            assert "overlaps" in lib.moe_last_error().decode()
    # Xc 512 bytes, Xs 32, Wc 8 KB, Ws 512, Y 2 KB
    good = [far, _at(2 << 20), _at(3 << 20), _at(4 << 20), offs]
    for i, size in enumerate((512, 32, 8192, 512, 20)):
        args = list(good)
        args[i] = _at(0)
        assert lib.moe_mx_grouped_forward(*args, 16, 4, 64, 64, 0, _at(size - size % 16 - 16 if size > 16 else 0), None) == capi.MOE_ERR_INVALID_ARG
        assert "overlaps" in lib.moe_last_error().decode()
    # 2 x 16 x 64 bf16 values: X 4 KB, codes 1 KB, scales 64 bytes
    for X, codes, scales in ((_at(0), _at(4080), far), (_at(0), far, _at(4080)), (far, _at(0), _at(1008))):
        assert lib.moe_mx_quantize(X, 0, 2, 16, 64, 2, codes, scales, None) == capi.MOE_ERR_INVALID_ARG
        assert "overlap" in lib.moe_last_error().decode()


# (gradient, result, values) of fp32 tensors; one with no values overlaps nothing
@pytest.mark.parametrize("tensors", [
    [(0, 0, 64), (0, 0, 64)],                             # the same gradient twice, in place
    [(4096, 4096, 64), (0, 0, 64), (252, 252, 64)],       # the last value of one is the first of another
    [(0, 4096, 64), (1024, 4348, 64)],                    # results
    [(0, 4096, 64), (4348, 8192, 64)],                    # a result and another gradient
    [(0, 4, 64)],                                         # a result and part of its own gradient
    [(4, 0, 64)],
    [(8192, 8192, 16), (0, 4096, 2000), (16384, 16384, 1)],  # a long result over a short one
    [(1 << 20, 4096, 64)],                                # the norm is a value of a gradient
    [(4096, 1 << 20, 64)],
    [(2 << 20, 4096, 64)],                                # the workspace
    [(4096, (2 << 20) + 8, 64)],
])
def test_clip_lists_that_overlap_are_refused(lib, tensors):
    need = ctypes.c_size_t()
    assert lib.moe_clip_workspace(len(tensors) + 1, ctypes.byref(need)) == capi.MOE_OK
    table = (capi.MoeGrad * (len(tensors) + 1))(capi.MoeGrad(_at(0), _at(0), 0, 1),
                                                *[capi.MoeGrad(_at(g), _at(o), n, 1) for g, o, n in tensors])
    status = lib.moe_clip_grad_norm(table, len(tensors) + 1, 1.0, _at(1 << 20), _at(2 << 20), need, None)
    assert status == capi.MOE_ERR_INVALID_ARG and "overlap" in lib.moe_last_error().decode()


@pytest.mark.parametrize("slices,rows,K,status", [
    (32, 2 ** 31 - 1, 32, capi.MOE_ERR_UNSUPPORTED),    # 2^31 blocks of rows
    (1, 2 ** 31 - 1, 32, capi.MOE_ERR_INVALID_ARG),     # a valid size: the missing pointer is refused
    (1, 1, 2 ** 31 - 32, capi.MOE_ERR_INVALID_ARG),
    (1, 2 ** 31 - 1, 2 ** 31 - 32, capi.MOE_ERR_UNSUPPORTED),
])
def test_mx_sizes_at_the_end_of_an_int(lib, slices, rows, K, status):
    assert lib.moe_mx_quantize(None, 0, slices, rows, K, 2, FAKE, FAKE, None) == status
    assert lib.moe_mx_dequantize(None, FAKE, 1, slices, rows, K, 0, FAKE, None) == status
    assert ("too large" in lib.moe_last_error().decode()) == (status == capi.MOE_ERR_UNSUPPORTED)


@pytest.mark.parametrize("at", [0, 959, 960, 961, 2000])
def test_clip_refuses_too_long_a_list_before_it_launches(lib, at):
    """More than 2^37 values among the tensors of one launch, wherever in the list they are."""
    n = 2100
    need = ctypes.c_size_t()
    assert lib.moe_clip_workspace(n, ctypes.byref(need)) == capi.MOE_OK
    for count in ((1 << 37) + 1, 1 << 62):
        table = (capi.MoeGrad * n)(*[capi.MoeGrad(_at(64 * i), _at(64 * i), 16, 1) for i in range(n)])
        table[at] = capi.MoeGrad(_at(1 << 40), _at(1 << 40), count, 0)
        assert lib.moe_clip_grad_norm(table, n, 1.0, _at(1 << 28), _at(1 << 29), need, None) == capi.MOE_ERR_UNSUPPORTED
        assert "2^37" in lib.moe_last_error().decode()
