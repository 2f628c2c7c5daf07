"""moe_clip_grad_norm at the ends of fp32's range, against fp64.

Tolerance: a thread's step sums up to 64 squares in four fp32 sums of 16 and adds those (18
roundings of 2^-24 of a sum of positive terms at most); pairs of fp32 numbers and fp64 follow.  The
square root halves that, the root is rounded: 10 * 2^-24 < 2^-20.  The factor adds the quotient's
rounding, a result the product's and its type's; results under the smallest normal value are off by
a subnormal step (two roundings of half of one)."""

import math

import pytest
import torch

from expert_routed_ffn_gb300 import capi

pytestmark = pytest.mark.gpu
REL = 2.0 ** -20


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_routed_ffn_gb300 import build
    build.build()
    capi.load()


def _norm(grads):
    return math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))


def _close(got, grad, factor):
    want = grad.double() * factor
    info = torch.finfo(got.dtype)
    slack = (REL + 2.0 ** -23 + info.eps / 2) * want.abs() + info.smallest_normal * info.eps
    assert bool(((got.double() - want).abs() <= slack).all())


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("value,max_norm", [
    (1e38, 1e-10), (1e38, 1e-3), (1e38, 0.7), (1e30, 1e-38), (1e38, 1e-38), (3e37, 1e-44),  # factors under 2^-126
    (1e-3, 1e-41), (1e-36, 1e-39), (1e-38, 2e-42),                                          # a subnormal max_norm
    (1e38, 1e30), (1e-30, 1e-33),
])
def test_factor_of_any_size(value, max_norm, dtype, inplace):
    gen = torch.Generator(device="cuda").manual_seed(81)
    grads = [(torch.rand(n, generator=gen, device="cuda") - 0.5).mul_(value).to(dtype) for n in (8192, 777, 3)]
    grads[1][5] = -value
    keep = [g.clone() for g in grads]
    out = grads if inplace else [torch.full_like(g, 9.0) for g in grads]
    norm = _norm(keep)
    got = float(capi.clip_grad_norm(grads, max_norm, out=None if inplace else out))
    if norm < torch.finfo(torch.float32).max:
        assert abs(got - norm) <= REL * norm + 2.0 ** -149
    limit = torch.tensor(max_norm, dtype=torch.float32).item()  # the argument is an fp32 number
    for o, k in zip(out, keep):
        _close(o, k, limit / norm)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("max_norm", [1.0, 1e-6, 1e38])
def test_norm_beyond_fp32(max_norm, dtype):
    """Finite gradients whose norm fp32 cannot hold: reported as an infinity, clipped by its value."""
    gen = torch.Generator(device="cuda").manual_seed(82)
    grads = [(torch.randint(0, 2, (n,), generator=gen, device="cuda") * 2 - 1).float().mul_(2e38).to(dtype) for n in (100_000, 77)]
    out = [torch.empty_like(g) for g in grads]
    assert float(capi.clip_grad_norm(grads, max_norm, out=out)) == float("inf")
    norm, limit = _norm(grads), torch.tensor(max_norm, dtype=torch.float32).item()
    assert math.isfinite(norm) and norm > torch.finfo(torch.float32).max
    for o, g in zip(out, grads):
        _close(o, g, limit / norm)
    assert float(capi.clip_grad_norm(grads, float("inf"), out=out)) == float("inf")  # the norm alone is wanted
    assert all(torch.equal(o, g) for o, g in zip(out, grads))
