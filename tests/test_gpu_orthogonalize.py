"""Orthogonalised updates (moe_orthogonalize) against fp64.

Bounds, derived before the first run, as 2-norms relative to the result's, u = 2^-12 (half a step of
fp16, a rounding's most; errors of a matrix of roundings add up like independent ones, which
2-norms of whole matrices measure).  Per step X, A and B are rounded once each.  B's roundings reach
X as E_B X (|E_B X| <= u |B|_F-like sums: each row of B X is off by u of the row's products), A's
through the polynomial's slope in A, at most |b| + 2 |c| 1.5 = 10.9: a step adds at most (1 + 10.9 / 2.8 + 1) u, taken
as 6 u; one step's error is carried into the next ones with at most the slope of the polynomial in X,
whose product over the last three steps is under 30 in the small directions and under 2 on the whole for
directions that have grown.  What is tested: 24 u for five steps where singular values fall off as
1 / sqrt(j) or slower, plus the result's own rounding (bf16: 2^-9 u-free).  For 16 directions 300 times
the rest the kept roundings leave those of the last two steps: the directions have grown by 3.4^3 = 39
by then, so u 300 / 39 = 8 u of noise, times 3.4^2 = 12: 96 u.
"""

import pytest
import torch

from expert_routed_ffn_gb300 import capi

pytestmark = pytest.mark.gpu

QUINTIC = (3.4445, -4.7750, 2.0315)
BF, F32 = torch.bfloat16, torch.float32
STEP = 2.0 ** -12


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_routed_ffn_gb300 import build
    build.build()
    capi.load()


@pytest.fixture(autouse=True)
def _status():
    yield
    assert capi.operators_status() == capi.MOE_OK


def _reference(G, coefficients, eps, scale=1.0):
    X = G.double()
    X = X / (X.flatten(-2).norm(dim=-1)[..., None, None] + eps)
    tall = X.shape[-2] > X.shape[-1]
    X = X.transpose(-1, -2) if tall else X
    for a, b, c in coefficients:
        A = X @ X.transpose(-1, -2)
        X = a * X + (b * A + c * A @ A) @ X
    return scale * (X.transpose(-1, -2) if tall else X)


def _gradient(E, N, K, dtype, seed=31, power=0.5):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = min(N, K)
    weight = torch.arange(1, r + 1, device="cuda", dtype=torch.float32) ** -power
    left = torch.randn(E, N, r, generator=gen, device="cuda") * weight
    G = left @ torch.randn(E, r, K, generator=gen, device="cuda") + torch.randn(E, N, K, generator=gen, device="cuda")
    return (1e-3 * G).to(dtype)


def _near(got, ref, units):
    """In each matrix of its own."""
    assert got.dtype == BF and got.shape == ref.shape and bool(torch.isfinite(got).all())
    ref, got = ref.reshape(-1, *ref.shape[-2:]), got.reshape(-1, *ref.shape[-2:])
    error = (got.double() - ref).flatten(1).norm(dim=1)
    bound = (units * STEP + 2.0 ** -8) * ref.flatten(1).norm(dim=1)
    assert bool((error <= bound).all()), float((error / ref.flatten(1).norm(dim=1)).max())


SIZES = [(1, 8, 8), (1, 64, 64), (3, 8, 200), (3, 200, 8), (2, 136, 264), (2, 264, 136), (1, 256, 1024), (1, 1024, 256), (5, 328, 328),
         (2, 520, 1032), (40, 256, 128), (1, 1408, 2048), (3, 2048, 1408), (130, 64, 72), (1, 4096, 264), (1, 264, 4096), (1, 64, 16384),
         (1, 16384, 64)]


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("E,N,K", SIZES)
def test_against_fp64(E, N, K, dtype):
    G = _gradient(E, N, K, dtype)
    out = torch.full((E, N, K), -3.0, dtype=BF, device="cuda")
    assert capi.orthogonalize(G, out=out) is out
    _near(out, _reference(G, [QUINTIC] * 5, 1e-7), 24)
    assert torch.equal(capi.orthogonalize(G), out)
    if E == 1:
        assert torch.equal(capi.orthogonalize(G[0]), out[0])


@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 8])
@pytest.mark.parametrize("N,K", [(136, 264), (264, 136)])
def test_steps_and_coefficients(N, K, steps):
    G = _gradient(2, N, K, F32)
    _near(capi.orthogonalize(G, steps=steps, scale=0.25), _reference(G, [QUINTIC] * steps, 1e-7, 0.25), 24)
    cubic = [(1.5, -0.5, 0.0)] * steps
    _near(capi.orthogonalize(G, steps=steps, coefficients=cubic), _reference(G, cubic, 1e-7), 24)
    mixed = [QUINTIC if i % 2 else (2.0, -1.5, 0.5) for i in range(steps)]
    _near(capi.orthogonalize(G, steps=steps, coefficients=mixed), _reference(G, mixed, 1e-7), 24)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,K", [(352, 512), (512, 352)])
def test_few_directions_far_above_the_rest(N, K, dtype):
    gen = torch.Generator(device="cuda").manual_seed(33)
    G = torch.randn(N, 16, generator=gen, device="cuda") @ torch.randn(16, K, generator=gen, device="cuda")
    G = (G + 0.05 * torch.randn(N, K, generator=gen, device="cuda")).to(dtype)
    _near(capi.orthogonalize(G), _reference(G, [QUINTIC] * 5, 1e-7), 96)


@pytest.mark.parametrize("factor", [1e-30, 1e-12, 1e25, 3e36])
def test_magnitudes(factor):
    """Squares beyond fp32 and below it; eps counts where the gradient is small."""
    G = _gradient(3, 72, 136, F32) * factor
    _near(capi.orthogonalize(G, eps=1e-30), _reference(G, [QUINTIC] * 5, 1e-30), 24)
    G[1] *= 1e-3  # every matrix by its own norm
    _near(capi.orthogonalize(G, eps=1e-30), _reference(G, [QUINTIC] * 5, 1e-30), 24)


def test_values_of_very_different_sizes():
    G = torch.zeros(2, 72, 136, device="cuda")
    G[0, 3, 5], G[1, 0, 0], G[1, 71, 135] = 2.0, 1e20, 1e20  # one and two directions
    _near(capi.orthogonalize(G), _reference(G, [QUINTIC] * 5, 1e-7), 24)


def test_zero_infinite_and_nan_matrices():
    G = _gradient(5, 72, 136, F32)
    want = capi.orthogonalize(G)
    G[0], G[2, 5, 7], G[3, 0, 0] = 0, float("inf"), float("nan")
    got = capi.orthogonalize(G)
    assert bool((got[0] == 0).all()) and bool(torch.isnan(got[2:4]).all())
    assert torch.equal(got[1], want[1]) and torch.equal(got[4], want[4])


def test_eps_beside_a_small_gradient():
    G = _gradient(1, 64, 128, F32)
    G = G / G.norm() * 3e-7
    _near(capi.orthogonalize(G, eps=1e-6), _reference(G, [QUINTIC] * 5, 1e-6), 24)


def test_in_place():
    G = _gradient(2, 136, 264, BF)
    for steps in (1, 2, 5):
        want = capi.orthogonalize(G, steps=steps)
        own = G.clone()
        assert capi.orthogonalize(own, steps=steps, out=own) is own and torch.equal(own, want)


def test_captured_and_on_another_stream():
    G = _gradient(4, 200, 328, F32)
    want = capi.orthogonalize(G)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = capi.orthogonalize(G, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = capi.orthogonalize(G)
    G.copy_(_gradient(4, 200, 328, F32, seed=34))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, capi.orthogonalize(G))


def test_wait_bound_of_zero_gives_up():
    lib = capi.load()
    G = _gradient(1, 64, 64, F32)
    try:
        assert lib.moe_operators_wait_limit(0) == capi.MOE_OK
        capi.orthogonalize(G)
        assert capi.operators_status() == capi.MOE_ERR_TIMEOUT
    finally:
        assert lib.moe_operators_wait_limit(-1) == capi.MOE_OK
    _near(capi.orthogonalize(G), _reference(G, [QUINTIC] * 5, 1e-7), 24)


def test_no_matrices_and_refusals():
    assert capi.orthogonalize(torch.empty(0, 64, 64, device="cuda")).shape == (0, 64, 64)
    G = _gradient(2, 64, 64, F32)
    for args in (dict(coefficients=[QUINTIC] * 4), dict(coefficients=(1.0, 2.0)), dict(out=G), dict(out=torch.zeros(2, 64, 32, dtype=BF, device="cuda")),
                 dict(G=G.half()), dict(G=G[:, :, ::2]), dict(G=G.cpu()), dict(G=G[0, 0])):
        with pytest.raises(ValueError):
            capi.orthogonalize(**{"G": G, **args})
    for args in (dict(steps=0, coefficients=[]), dict(eps=0.0), dict(scale=float("inf")), dict(coefficients=(float("nan"), 0.0, 0.0)),
                 dict(coefficients=(1e6, 1.0, 1.0)), dict(G=torch.zeros(2, 12, 64, device="cuda"))):
        with pytest.raises(capi.MoeError):
            capi.orthogonalize(**{"G": G, **args})
    base = torch.zeros(64 * 64 + 64, dtype=BF, device="cuda")
    with pytest.raises(capi.MoeError):  # in place, but shifted
        capi.orthogonalize(base[:4096].view(64, 64), out=base[64:].view(64, 64))
