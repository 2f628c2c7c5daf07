"""What moe_orthogonalize's roundings cost, against the same chain of roundings in 64 bits.

The kernel rounds X, A and B to fp16 once a step and carries the low half of X through a X in all steps but the
last two; products are summed in fp32.  `_chain` does the same in 64 bits, from the description in include/moe.h.
Both errors (2-norm, against the chain without roundings) are root sums of squares over more than 10^4 independent
roundings of the same sizes, equal within a few percent; fp32 sums add at most 2^-13 of a step's result, which
grows like the other roundings do.  So the kernel may be 1.25 times as far off as `_chain`.

That the bound tells a lost low half from a kept one is shown on the CPU, with the mistakes planted in
`_chain`: with 16 directions 300 times the others they cost 2.4 times the error and more.
"""

import pytest
import torch

BF, F32 = torch.bfloat16, torch.float32
QUINTIC = (3.4445, -4.7750, 2.0315)
CUBIC = (1.5, -0.5, 0.0)
FACTOR = 1.25


def _half(x, scale):
    return (x * scale).float().half().double() / scale


def _carried(step, steps):
    return step < steps - 2


def _chain(G, coefficients, rounded=True, carried=_carried, low_of_first=True, eps=1e-7):
    """The iteration in 64 bits; rounded: with the kernel's roundings."""
    X = G.double()
    X = X / (X.norm() + eps)
    tall = X.shape[0] > X.shape[1]
    X = X.t() if tall else X
    n, eye = len(coefficients), torch.eye(X.shape[0], dtype=torch.float64, device=G.device)
    keep = (lambda v, scale: _half(v, scale)) if rounded else (lambda v, scale: v)
    low = 0 * X
    if rounded and G.dtype == F32:  # (bf16 values are exact in fp16)
        low = X - _half(X, 2.0 ** 12)
        X = X - low
        low = _half(low, 2.0 ** 12) if low_of_first and carried(0, n) else 0 * X
    for i, (a, b, c) in enumerate(coefficients):
        A = keep(X @ X.t(), 2.0 ** 13)
        B = keep(a * eye + b * A + c * A @ A, 2.0 ** 12)
        Y = B @ X + a * low
        if i + 1 == n:
            X = Y
            break
        X = keep(Y, 2.0 ** 12)
        low = _half(Y - X, 2.0 ** 12) if carried(i + 1, n) else 0 * X
    X = X.t() if tall else X
    return X.to(BF).double() if rounded else X


def _error(got, ref):
    return float((got.double() - ref).norm() / ref.norm())


def _few(N, K, dtype, seed=33, device="cpu"):
    """16 directions 300 times as large as the others."""
    gen = torch.Generator().manual_seed(seed)
    G = torch.randn(N, 16, generator=gen) @ torch.randn(16, K, generator=gen) + 0.05 * torch.randn(N, K, generator=gen)
    return G.to(dtype).to(device)


def _falling(N, K, dtype, seed=34, device="cpu"):
    gen = torch.Generator().manual_seed(seed)
    r = min(N, K)
    G = (torch.randn(N, r, generator=gen) * torch.arange(1, r + 1) ** -0.5) @ torch.randn(r, K, generator=gen) + torch.randn(N, K, generator=gen)
    return (1e-3 * G).to(dtype).to(device)


MISTAKES = {
    "no low half": dict(carried=lambda i, n: False),
    "the first one alone": dict(carried=lambda i, n: i == 0),
    "one step too few": dict(carried=lambda i, n: i < n - 3),
    "not of the gradient itself": dict(low_of_first=False),
}


@pytest.mark.parametrize("mistake", list(MISTAKES))
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,K", [(352, 512), (512, 352)])
def test_the_bound_tells_a_lost_low_half(N, K, dtype, mistake):
    if mistake == "not of the gradient itself" and dtype == BF:
        pytest.skip("bf16 gradients have no low half")
    G = _few(N, K, dtype)
    ref = _chain(G, [QUINTIC] * 5, rounded=False)
    kept = _error(_chain(G, [QUINTIC] * 5), ref)
    lost = _error(_chain(G, [QUINTIC] * 5, **MISTAKES[mistake]), ref)
    assert kept <= 2.5e-3 and lost > 2.0 * kept > FACTOR * kept, (kept, lost)


def test_errors_that_the_header_states():
    """What include/moe.h says of the quintic's steps (8: of smaller matrices too), and of an iteration that converges."""
    for G in (_few(264, 352, F32), _falling(264, 352, F32), _falling(264, 352, BF, seed=3)):
        for steps, stated in ((5, 2.3e-3), (6, 2.6e-3), (8, 3.1e-3), (20, 7e-3), (64, 3e-2)):
            assert _error(_chain(G, [QUINTIC] * steps), _chain(G, [QUINTIC] * steps, rounded=False)) <= stated
            assert _error(_chain(G, [CUBIC] * steps), _chain(G, [CUBIC] * steps, rounded=False)) <= 2e-3


@pytest.fixture
def capi():
    from expert_routed_ffn_gb300 import build, capi
    build.build()
    capi.load()
    yield capi
    assert capi.operators_status() == capi.MOE_OK


def _held(capi, G, coefficients, **how):
    ref = _chain(G, coefficients, rounded=False, **how)
    bound = FACTOR * _error(_chain(G, coefficients, **how), ref)
    got = _error(capi.orthogonalize(G, steps=len(coefficients), coefficients=coefficients, **how), ref)
    print(f"{got:.3e} of {bound:.3e}")
    assert got <= bound, (got, bound)
    return got


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,K", [(352, 512), (512, 352), (1032, 2056), (264, 4096)])
@pytest.mark.parametrize("seed", [33, 35])
def test_few_directions_far_above_the_rest(capi, N, K, dtype, seed):
    assert _held(capi, _few(N, K, dtype, seed, "cuda"), [QUINTIC] * 5) <= 2.8e-3


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("N,K", [(352, 512), (512, 352), (1408, 2048), (224, 96)])
def test_falling_singular_values(capi, N, K, dtype):
    assert _held(capi, _falling(N, K, dtype, device="cuda"), [QUINTIC] * 5) <= 2.5e-3


@pytest.mark.gpu
@pytest.mark.parametrize("steps", [1, 2, 3, 4, 6, 8, 12, 20, 64])
@pytest.mark.parametrize("triple", [QUINTIC, CUBIC])
def test_steps(capi, steps, triple):
    for G in (_few(264, 352, F32, device="cuda"), _falling(352, 264, BF, device="cuda")):
        _held(capi, G, [triple] * steps)
