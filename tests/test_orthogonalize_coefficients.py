"""Coefficients under which X or the polynomial would leave what fp16 holds are refused, on the host; the others
reach the GPU."""

import ctypes

import pytest

from expert_routed_ffn_gb300 import build as moe_build
from expert_routed_ffn_gb300 import capi

QUINTIC = (3.4445, -4.7750, 2.0315)


@pytest.fixture(scope="module")
def lib():
    moe_build.build()
    return capi.load()


def _status(lib, triples, E):
    table = (ctypes.c_float * (3 * len(triples)))(*[v for t in triples for v in t])
    return lib.moe_orthogonalize(None, 1, E, 64, 64, table, len(triples), 1e-7, 1.0, None, None, 0, None)


@pytest.mark.parametrize("triples", [
    [(0.0, 0.0, 0.0)], [(1e-6, 0.0, 0.0)], [(5e-4, 0.0, 0.0)], [QUINTIC, (1e-4, 0.0, 0.0)],  # a polynomial of nearly nothing
    [(0.0009, 0.0, 0.0), QUINTIC], [(0.01, 0.0, 0.0), (0.01, 0.0, 0.0), QUINTIC],  # singular values that vanish
    [(2000.0, 0.0, 0.0)], [(40.0, 0.0, 0.0), (40.0, 0.0, 0.0)], [(1.0, 1e30, 0.0)],  # and that grow
])
def test_refused(lib, triples):
    assert _status(lib, triples, 0) == capi.MOE_ERR_UNSUPPORTED
    assert "singular values" in lib.moe_last_error().decode()


@pytest.mark.parametrize("triples", [[QUINTIC] * 5, [QUINTIC] * 64, [(1.5, -0.5, 0.0)] * 20, [(15 / 8, -10 / 8, 3 / 8)], [(1.0, 0.0, 0.0)],
                                     [(0.0, 1.0, 0.0)], [(0.0, 0.0, 1.0)] * 2, [(0.01, 0.0, 0.0), (50.0, 0.0, 0.0)], [(30.0, 0.0, 0.0), (30.0, 0.0, 0.0)]])
def test_accepted(lib, triples):
    assert _status(lib, triples, 0) == capi.MOE_OK  # no matrices: nothing to do
    assert _status(lib, triples, 1) == capi.MOE_ERR_INVALID_ARG  # NULL pointers


@pytest.mark.gpu
@pytest.mark.parametrize("triples", [[(0.002, 0.0, 0.0)], [(0.01, 0.0, 0.0), (50.0, 0.0, 0.0)], [(30.0, 0.0, 0.0), (30.0, 0.0, 0.0)],
                                     [(900.0, 0.0, 0.0), (0.002, 0.0, 0.0), (1.0, 0.0, 0.0)], [(0.0, 1.0, 0.0)]])
@pytest.mark.parametrize("N,K", [(72, 136), (1032, 512)])
def test_the_ends_of_what_is_accepted(lib, triples, N, K):
    """Five roundings of 2^-12 a step (X, A and the polynomial; A counts twice in X A and A X), as 2-norms, and the result's."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(43)
    G = torch.randn(N, K, generator=gen, device="cuda")
    X = G.double() / (G.double().norm() + 1e-7)
    for a, b, c in triples:
        A = X @ X.t()
        X = a * X + (b * A + c * A @ A) @ X
    got = capi.orthogonalize(G, steps=len(triples), coefficients=triples).double()
    assert float((got - X).norm()) <= (5 * len(triples) * 2.0 ** -12 + 2.0 ** -8) * float(X.norm())
    assert capi.operators_status() == capi.MOE_OK
