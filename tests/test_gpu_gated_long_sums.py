"""The gated products whose sums come in several segments for bf16 results: more than 16384 products.

Operands of one sign, where the tensor core's truncation shows most.  A segment's 1024 instructions lose up to
2^-23 of its sum each, 2^-13; the sums of segments, to nearest, 2^-24 of the whole each.  Then one rounding."""

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
    yield
    assert capi.operators_status() == capi.MOE_OK


@pytest.mark.parametrize("I", [8192, 8200, 12296, 20480])  # 2 I products: one segment, and more, whole or not
@pytest.mark.parametrize("counts,before,behind", [([1, 0, 37, 64], 3, 5), ([300, 1, 513], 0, 0), ([20] * 40, 0, 1)])
@pytest.mark.parametrize("signs", [False, True])
def test_dgrad(I, counts, before, behind, signs):
    K, E, rows = 136, len(counts), before + sum(counts) + behind
    gen = torch.Generator(device="cuda").manual_seed(95)

    def bf(*shape):
        t = torch.randn(*shape, generator=gen, device="cuda")
        return (t if signs else t.abs()).to(BF)

    dG, dU, Wg, Wu = bf(rows, I), bf(rows, I), bf(E, I, K), bf(E, I, K)
    ends = [before]
    for n in counts:
        ends.append(ends[-1] + n)
    offs = torch.tensor(ends, dtype=torch.int32, device="cuda")
    out = torch.full((rows, K), -3.0, dtype=BF, device="cuda")
    capi.grouped_gated_dgrad(dG, dU, Wg, Wu, offs, out=out)
    assert bool((out[:before] == -3.0).all()) and bool((out[ends[-1]:] == -3.0).all())
    segments = -(-2 * (-(-I // 64) * 64) // 16384)
    for e in range(E):
        r = slice(ends[e], ends[e + 1])
        parts = [(a[r].double(), w[e].double()) for a, w in ((dG, Wg), (dU, Wu))]
        ref = sum(a @ w for a, w in parts)
        bound = (2.0 ** -13 + segments * 2.0 ** -24) * sum(a.abs() @ w.abs() for a, w in parts)
        bound = bound + 2.0 ** -8 * (ref.abs() + bound)
        assert bool(((out[r].double() - ref).abs() <= bound).all()), float(((out[r].double() - ref).abs() / bound).max())
    again = capi.grouped_gated_dgrad(dG, dU, Wg, Wu, offs)
    assert torch.equal(again[before:ends[-1]], out[before:ends[-1]])
