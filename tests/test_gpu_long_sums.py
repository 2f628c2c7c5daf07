"""Long sums of the grouped products: bf16 results, accumulation and MXFP4 operands.

The tensor core truncates as it adds.  An instruction's addition loses at most 2^-23 of the running
sum, so n of them, of products of one sign (the worst case), lose on average half of n 2^-23 of the
result; a factor of two is left for the order of the products within an instruction.  One
accumulator takes 256 additions (fp32 results) or 1024 (bf16), whatever the length of the sum, and
segments are added to nearest (64 of them: 2^-18 at most): the bound does not grow with the length.
A bf16 result is rounded once, by at most 2^-8 of its value; over the elements that rounding is
even, so their mean shows what the sums lost."""

import pytest
import torch

from expert_routed_ffn_gb300 import capi

pytestmark = pytest.mark.gpu
LOSS = {torch.float32: 2.0 ** -15 + 2.0 ** -18, torch.bfloat16: 2.0 ** -13 + 2.0 ** -18}


@pytest.fixture(scope="module", autouse=True)
def _built():
    from expert_routed_ffn_gb300 import build
    build.build()
    capi.load()


@pytest.fixture(autouse=True)
def _status():
    yield
    assert capi.operators_status() == capi.MOE_OK


def _offs(counts):
    return torch.tensor([0] + [sum(counts[:i + 1]) for i in range(len(counts))], dtype=torch.int32, device="cuda")


def _positive(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda").abs().to(torch.bfloat16)


def _check(got, ref):
    """got against a reference > 0 in fp64"""
    rel = (got.double() - ref) / ref
    loss = LOSS[got.dtype]
    half = torch.finfo(got.dtype).eps / 2 if got.dtype == torch.bfloat16 else 0.0
    assert float(rel.abs().max()) <= loss + half * (1 + loss)
    # rounding errors spread over [-half, half]: their mean is within 6 of its deviations of zero
    assert abs(float(rel.mean())) <= loss + 6 * half / (3 * rel.numel()) ** 0.5


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts", [[70, 0, 33, 1], [300, 500]])
@pytest.mark.parametrize("length", [16392, 65536, 262152])
@pytest.mark.parametrize("op", ["forward", "dgrad"])
def test_products_over_a_long_axis(op, length, counts, dtype):
    gen = torch.Generator(device="cuda").manual_seed(71)
    n = 1032  # with 300 and 500 rows a CTA pair may take more than one tile
    A = _positive(gen, sum(counts), length)
    W = _positive(gen, len(counts), *((n, length) if op == "forward" else (length, n)))
    call = capi.grouped_forward if op == "forward" else capi.grouped_dgrad
    got = call(A, W, _offs(counts), out_dtype=dtype)
    ref, at = torch.empty(got.shape, dtype=torch.float64, device="cuda"), 0
    for e, c in enumerate(counts):
        w = W[e].t() if op == "forward" else W[e]
        ref[at:at + c] = sum(A[at:at + c, k:k + 32768].double() @ w[k:k + 32768].double() for k in range(0, length, 32768))
        at += c
    _check(got, ref)
    assert torch.equal(call(A, W, _offs(counts), out_dtype=dtype), got)


# sums of one, of some and of many segments behind one another, in every order; tails of every kind
ROWS = {"few": [262_145, 3], "mixed": [16_384, 0, 16_385, 5, 40_016, 65_535, 70, 16_400, 33_000, 1, 0, 50_001]}


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("size", [(136, 264), (1024, 1032)])
@pytest.mark.parametrize("name", list(ROWS))
def test_weight_gradients_of_many_rows(name, size, dtype, accumulate):
    gen = torch.Generator(device="cuda").manual_seed(72)
    counts = ROWS[name]
    dY, X, offs = _positive(gen, sum(counts), size[0]), _positive(gen, sum(counts), size[1]), _offs(counts)
    first, at, ref = torch.ones((len(counts),) + size, dtype=dtype, device="cuda"), 0, []
    for c in counts:
        ref.append(sum((dY[r:min(r + 32768, at + c)].double().t() @ X[r:min(r + 32768, at + c)].double()
                        for r in range(at, at + c, 32768)), torch.zeros(size, dtype=torch.float64, device="cuda")))
        at += c
    ref = torch.stack(ref)
    out = first.clone()
    assert capi.grouped_wgrad(dY, X, offs, out=out, accumulate=accumulate) is out
    if accumulate:
        ref += 1
    empty = [e for e, c in enumerate(counts) if c == 0]
    assert torch.equal(out[empty], first[empty] * accumulate)
    for e, c in enumerate(counts):
        if c:
            _check(out[e], ref[e])
    again = first.clone()
    assert torch.equal(capi.grouped_wgrad(dY, X, offs, out=again, accumulate=accumulate), out)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("counts,N", [([40, 0, 33, 7], 144), ([300, 5, 500], 1032), ([512, 1024], 528)])
@pytest.mark.parametrize("length", [16416, 65536, 262176])
def test_mxfp4_products_over_a_long_axis(length, counts, N, dtype):
    """Blocks whose magnitudes differ by powers of two, so that sums do not fit fp32 exactly."""
    gen = torch.Generator(device="cuda").manual_seed(73)

    def tensor(*shape):
        spread = torch.randint(-6, 7, shape[:-1] + (shape[-1] // 32,), generator=gen, device="cuda")
        x = torch.randn(shape, generator=gen, device="cuda").abs()
        return x.unflatten(-1, (-1, 32)).mul_(torch.exp2(spread.float()).unsqueeze(-1)).flatten(-2)

    X, W = (capi.mx_quantize(tensor(*s), "mxfp4") for s in ((sum(counts), length), (len(counts), N, length)))
    offs = _offs(counts)
    got = capi.mx_grouped_forward(*X, *W, offs, out_dtype=dtype)
    x, ref, at = capi.mx_dequantize(*X, "mxfp4", torch.float32), torch.empty(got.shape, dtype=torch.float64, device="cuda"), 0
    for e, c in enumerate(counts):
        w = capi.mx_dequantize(W[0][e].clone(), W[1][e].clone(), "mxfp4", torch.float32).t()
        ref[at:at + c] = sum(x[at:at + c, k:k + 32768].double() @ w[k:k + 32768].double() for k in range(0, length, 32768))
        at += c
    _check(got, ref)
    assert torch.equal(capi.mx_grouped_forward(*X, *W, offs, out_dtype=dtype), got)
