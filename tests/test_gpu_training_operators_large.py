"""The training operators where tensors pass 2^31 values and 2^32 bytes: the last rows and matrices are
what a call on them alone gives.  A row's (a matrix's) sums have one order whatever the call's size, so
the norms give the same bits; the products' tiles differ with it, so they are held to fp64."""

import pytest
import torch

from expert_routed_ffn_gb300 import capi

pytestmark = pytest.mark.gpu

BF = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_routed_ffn_gb300 import build
    build.build()
    capi.load()


@pytest.fixture(autouse=True)
def _status():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()
    assert capi.operators_status() == capi.MOE_OK


def _ends(n, k=300):
    """The first and the last k rows."""
    return torch.cat([torch.arange(k), torch.arange(n - k, n)]).cuda()


def test_norms():
    T, H = 300_000, 8192
    gen = torch.Generator(device="cuda").manual_seed(51)
    one = torch.randn(1000, H, generator=gen, device="cuda").to(BF)
    X = one.repeat(T // 1000, 1)
    F = one.flip(0).repeat(T // 1000, 1)
    X[-7:], F[-5:] = 3.0, -2.0  # the last rows are like no others
    how = dict(pre_w=torch.rand(H, generator=gen, device="cuda"), post_w=torch.rand(H, generator=gen, device="cuda"))
    at = _ends(T)
    new, N = capi.sandwich_norm(X, F, **how)
    want = capi.sandwich_norm(X[at], F[at], **how)
    assert torch.equal(new[at], want[0]) and torch.equal(N[at], want[1])
    back = capi.sandwich_norm_backward(F, X, new, F, **how)
    part = capi.sandwich_norm_backward(F[at], X[at], new[at], F[at], **how)
    assert torch.equal(back[0][at], part[0]) and torch.equal(back[1][at], part[1])


def test_gated_products():
    rows, E, I, K = 1_050_000, 3, 2056, 72
    gen = torch.Generator(device="cuda").manual_seed(52)
    X = torch.randn(1000, K, generator=gen, device="cuda").to(BF).repeat(rows // 1000, 1)
    X[-7:] = 0.25
    Wg, Wu = (torch.randn(E, I, K, generator=gen, device="cuda").mul_(0.1).to(BF) for _ in range(2))
    offs = torch.tensor([0, 11, rows - 200, rows], dtype=torch.int32, device="cuda")
    H, G, U = capi.grouped_gated_forward(X, Wg, Wu, offs, save=True)
    at = torch.arange(rows - 150, rows, device="cuda")  # of the last expert
    x, wg, wu = X[at].double(), Wg[2].double(), Wu[2].double()
    g, u = x @ wg.t(), x @ wu.t()
    # a rounding to bf16 each (2^-9 of a value at most, 2^-8 with what the fp32 sums add)
    for got, want in ((G, g), (U, u), (H, g * torch.sigmoid(g) * u)):
        assert float((got[at].double() - want).norm()) <= 2.0 ** -8 * float(want.norm())
    Wd = torch.randn(E, K, I, generator=gen, device="cuda").mul_(0.1).to(BF)
    dG, dU = capi.grouped_gated_backward(X, Wd, G, U, offs)
    dh, s = x @ Wd[2].double(), torch.sigmoid(G[at].double())
    want = dh * G[at].double() * s
    assert float((dU[at].double() - want).norm()) <= 2.0 ** -8 * float(want.norm())
    dX = capi.grouped_gated_dgrad(dG, dU, Wg, Wu, offs, out_dtype=torch.float32)
    want = dG[at].double() @ wg + dU[at].double() @ wu
    assert float((dX[at].double() - want).norm()) <= 2.0 ** -12 * float(want.norm())  # 4112 products in fp32


def test_orthogonalised_updates():
    E, N, K = 1030, 1024, 2056
    gen = torch.Generator(device="cuda").manual_seed(53)
    G = torch.empty(E, N, K, dtype=BF, device="cuda")
    for e in range(E):
        G[e] = torch.randn(N, K, generator=gen, device="cuda")
    out = capi.orthogonalize(G, steps=3)
    for e in (0, 517, E - 1):
        X = G[e].double()
        X = X / (X.norm() + 1e-7)
        for _ in range(3):
            A = X @ X.t()
            X = 3.4445 * X + (-4.7750 * A + 2.0315 * A @ A) @ X
        # the bound of tests/test_gpu_orthogonalize.py
        assert float((out[e].double() - X).norm()) <= (24 * 2.0 ** -12 + 2.0 ** -8) * float(X.norm())
