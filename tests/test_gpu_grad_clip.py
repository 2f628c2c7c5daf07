"""moe_clip_grad_norm against fp64.

Tolerance: a thread sums 32 squares in fp32 (at most 34 roundings of 2^-24 of the sum, all
terms positive), the rest is fp64; the square root halves the relative error and the norm is
rounded once: (34 / 2 + 1) * 2^-24 < 2^-19.  A clipped value: the factor's rounding and the
norm's error (no more than 18 * 2^-24 together), the product's rounding, the output type's."""

import math

import pytest
import torch

from expert_routed_ffn_gb300 import capi

pytestmark = pytest.mark.gpu
REL = 2.0 ** -19


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_routed_ffn_gb300 import build
    build.build()
    capi.load()


def _tensors(sizes, kinds, std=1.0, seed=31):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    return [(torch.randn(n, generator=gen, device="cuda") * std * (1 + i % 3)).to(kinds[i % len(kinds)])
            for i, n in enumerate(sizes)]


def _norm(grads):
    return math.sqrt(sum(float((g.double() ** 2).sum()) for g in grads))


def _close(got, grad, factor):
    want = grad.double() * factor
    # products under the smallest normal value are off by half a subnormal step instead
    slack = (REL + 2.0 ** -24 + torch.finfo(got.dtype).eps / 2) * want.abs() + torch.finfo(got.dtype).smallest_normal * torch.finfo(got.dtype).eps
    assert bool(((got.double() - want).abs() <= slack).all())


LISTS = {
    "one_value": [1],
    "odd": [1, 7, 8191, 8192, 8193, 3, 100_001],
    "with_empty": [0, 5, 0, 8192, 0],
    "many": [1 + (37 * i) % 1500 for i in range(700)],
    "over_one_launch": [1 + i % 60 for i in range(2100)],
    "large": [30_000_001, 20_000_000],
}


@pytest.mark.parametrize("inplace", [True, False])
@pytest.mark.parametrize("kinds", [(torch.float32,), (torch.bfloat16,), (torch.bfloat16, torch.float32)])
@pytest.mark.parametrize("name", list(LISTS))
def test_against_fp64(name, kinds, inplace):
    grads = _tensors(LISTS[name], kinds)
    norm = _norm(grads)
    for share in (0.3, 4.0):
        work = [g.clone() for g in grads]
        out = None if inplace else [torch.full_like(g, 9.0) for g in grads]
        got = capi.clip_grad_norm(work, share * norm, out=out)
        assert got.dtype == torch.float32 and got.dim() == 0
        assert abs(float(got) - norm) <= REL * norm
        for g, w, o in zip(grads, work, work if inplace else out):
            if share > 1:
                assert torch.equal(o, g)
            else:
                _close(o, g, share)
            if not inplace:
                assert torch.equal(w, g)
        again = [g.clone() for g in grads]
        assert torch.equal(capi.clip_grad_norm(again, share * norm), got)  # the same order of sums every time
        assert all(torch.equal(a, o) for a, o in zip(again, work if inplace else out))


def test_unaligned_views():
    flat = torch.randn(50_000, device="cuda")
    half = torch.randn(50_000, device="cuda").to(torch.bfloat16)
    keep = flat.clone(), half.clone()
    grads = [flat[1:20_000], flat[20_003:49_999], half[1:10_000], half[10_001:49_001]]
    ref = [g.clone() for g in grads]
    norm = _norm(ref)
    assert abs(float(capi.clip_grad_norm(grads, norm / 2)) - norm) <= REL * norm
    for g, r in zip(grads, ref):
        _close(g, r, 0.5)
    for t, k, untouched in ((flat, keep[0], [0, 20_000, 20_002, 49_999]), (half, keep[1], [0, 10_000, 49_001])):
        assert all(t[i] == k[i] for i in untouched)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e19, 1e25])
def test_squares_beyond_fp32(scale, dtype):
    grads = _tensors([8192, 777], (dtype,), std=scale)
    norm = _norm(grads)
    assert abs(float(capi.clip_grad_norm([g.clone() for g in grads], 1e38)) - norm) <= REL * norm
    out = [torch.empty_like(g) for g in grads]
    capi.clip_grad_norm(grads, norm / 8, out=out)
    for o, g in zip(out, grads):
        _close(o, g, 1 / 8)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_gradients_pass_through(bad):
    grads = _tensors([9000, 50], (torch.float32, torch.bfloat16))
    grads[1][7] = bad
    out = [torch.zeros_like(g) for g in grads]
    norm = capi.clip_grad_norm(grads, 1.0, out=out)
    assert not math.isfinite(float(norm)) and math.isnan(float(norm)) == math.isnan(bad)
    for g, o in zip(grads, out):
        assert torch.equal(g.nan_to_num(nan=5.0), o.nan_to_num(nan=5.0))


def test_zero_gradients_and_infinite_limit():
    grads = [torch.zeros(5000, device="cuda"), torch.zeros(3, device="cuda", dtype=torch.bfloat16)]
    assert float(capi.clip_grad_norm(grads, 0.1)) == 0.0
    g = torch.full((4,), 3.0, device="cuda")
    assert float(capi.clip_grad_norm([g], float("inf"))) == 6.0 and bool((g == 3).all())


def test_long_tensor():
    """More than 2^31 values in one tensor."""
    if torch.cuda.get_device_properties(0).total_memory < 40e9:
        pytest.skip("needs 40 GB")
    g = torch.zeros(2_200_000_005, dtype=torch.bfloat16, device="cuda")
    g[-5:] = 3.0
    g[0] = 2.0
    assert abs(float(capi.clip_grad_norm([g], 0.7)) - 7.0) <= 7 * REL
    assert abs(float(g[-1]) - 0.3) < 2e-3 and abs(float(g[0]) - 0.2) < 2e-3


def test_captured_and_two_streams():
    a, b = _tensors([40_000, 9], (torch.float32,)), _tensors([40_000, 9], (torch.bfloat16,), seed=32)
    oa, ob = [torch.empty_like(g) for g in a], [torch.empty_like(g) for g in b]
    graphs = []
    for grads, out in ((a, oa), (b, ob)):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            norm = capi.clip_grad_norm(grads, 1.0, out=out)
        graphs.append((graph, norm))
    for g in a + b:
        g.mul_(2)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for _ in range(4):
        for (graph, _), s in zip(graphs, streams):  # each has a workspace of its own
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (_, norm), grads, out in ((graphs[0], a, oa), (graphs[1], b, ob)):
        want = _norm(grads)
        assert abs(float(norm) - want) <= REL * want
        for o, g in zip(out, grads):
            _close(o, g, 1 / want)


def test_refusals():
    g = torch.zeros(8, device="cuda")
    with pytest.raises(ValueError, match="at least one"):
        capi.clip_grad_norm([], 1.0)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        capi.clip_grad_norm([g.half()], 1.0)
    with pytest.raises(ValueError, match="contiguous"):
        capi.clip_grad_norm([torch.zeros(4, 4, device="cuda").t()], 1.0)
    with pytest.raises(ValueError, match="device"):
        capi.clip_grad_norm([g.cpu()], 1.0)
    with pytest.raises(ValueError, match="device"):
        capi.clip_grad_norm([g, g.cpu()], 1.0)
    with pytest.raises(ValueError, match="each"):
        capi.clip_grad_norm([g], 1.0, out=[g, g])
    with pytest.raises(ValueError, match="types and sizes"):
        capi.clip_grad_norm([g], 1.0, out=[g[:4]])
    for bad in (0.0, -1.0, float("nan")):
        with pytest.raises(capi.MoeError, match="max_norm"):
            capi.clip_grad_norm([g], bad)


def test_gradients_that_touch_or_repeat():
    """Neighbours in one buffer, in any order, are no overlap; nor are inputs that repeat."""
    flat = _tensors([50_000], (torch.float32,))[0]
    ref, cuts = flat.clone(), [0, 1, 9000, 20_003, 50_000]
    parts = [flat[a:b] for a, b in zip(cuts, cuts[1:])]
    norm = _norm([flat])
    assert abs(float(capi.clip_grad_norm([parts[i] for i in (2, 0, 3, 1)], norm / 2)) - norm) <= REL * norm
    _close(flat, ref, 0.5)
    out = [torch.empty_like(ref), torch.empty_like(ref)]
    got = capi.clip_grad_norm([ref, ref], norm / 2, out=out)
    assert abs(float(got) - 2 ** 0.5 * norm) <= REL * 2 ** 0.5 * norm
    assert torch.equal(out[0], out[1])
    _close(out[0], ref, 0.5 ** 1.5)
    for grads, into in (([ref, ref], None), ([ref], [ref[1:]]), ([ref[1:], flat], [flat[1:], out[0]])):
        with pytest.raises((capi.MoeError, ValueError), match="overlap|sizes"):
            capi.clip_grad_norm(grads, 1.0, out=into)
